// norm_rope.cu -- what sits between the projections and the chunked attention,
// in one pass over the data: the RMS norm of every query and key head, the
// rotary position of the row, and the write of the chunk's keys and values
// into the caches; and its backward.
//
//   forward, per (row, head), x [d]:
//     r = 1 / sqrt(mean x^2 + eps),  n = r gamma o x   (n = x without a norm)
//     pair (a, b) of n at angle t:   (a cos t - b sin t, b cos t + a sin t)
//   backward, from dy (float32 from the attention):
//     dn = dy rotated by -t
//     dx = r (gamma o dn - xhat mean(gamma o dn o xhat)),  xhat = r x
//     dgamma += sum over rows and heads of dn o xhat
//
// The angle of pair i at position p is p f_i.  Float32 loses it for positions
// in the tens of thousands, and float64 is slow on this GPU, so the frequency
// is held in turns as a 64-bit fixed-point fraction: p * turns_i mod 2^64 is
// the exact fraction of a turn, whatever p, with one integer multiplication;
// it is rounded to float32 once and goes to sincospi.
//
// One warp takes a row (all of its heads, or a share of them when there are
// few rows): eight elements a lane, d / 8 lanes a head, 32 / (d / 8) heads at
// a time.  A lane's cosines and sines belong to its element indices, so they
// are computed once a row and reused for every head; the partner of a
// half-split pair sits rot / 16 lanes away (a shuffle), that of an interleaved
// pair in the same lane.  Bound by HBM: every element is read and written once.
#include <cuda_bf16.h>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace seqattn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

template <typename E>
__device__ __forceinline__ void load8(const E* p, float (&f)[8]) {
  if constexpr (sizeof(E) == 2) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

template <typename E>
__device__ __forceinline__ void store8(E* p, const float (&f)[8]) {
  if constexpr (sizeof(E) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// Sum over the LPH lanes of a head (every lane gets it; same order everywhere).
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The rotation as this lane sees it: y[i] = x[i] c[i] + partner(x)[i] s[i].
struct Rotation {
  float c[8], s[8];
  int src;            // lane that holds the partners (half-split); own lane if none
  bool inter;
};

// `l`: lane within the head, `sign` +1 forward, -1 backward.
template <int LPH>
__device__ __forceinline__ void set_rotation(Rotation& rt, const NormRopeParams& p, int l, int lane, int64_t row,
                                             int64_t pos0, float sign) {
  const int e0 = 8 * l;
  const int half = p.rot_dim / 2;
  rt.src = lane;
  rt.inter = p.interleaved != 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) rt.c[i] = 1.f, rt.s[i] = 0.f;
  if (e0 >= p.rot_dim) return;
  const int64_t rows = static_cast<int64_t>(p.B) * p.q_len;
  if (rt.inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = e0 / 2 + i;
      const int64_t pos = p.positions ? p.positions[p.axis[pair] * rows + row] : pos0;
      const float turn2 = __ll2float_rn(static_cast<long long>(static_cast<uint64_t>(pos) * p.turns[pair])) * 0x1p-63f;
      float sn, cs;
      sincospif(turn2, &sn, &cs);
      rt.c[2 * i] = rt.c[2 * i + 1] = cs;
      rt.s[2 * i] = -sign * sn;
      rt.s[2 * i + 1] = sign * sn;
    }
  } else {
    const bool first = e0 < half;
    rt.src = first ? lane + half / 8 : lane - half / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = (first ? e0 : e0 - half) + i;
      const int64_t pos = p.positions ? p.positions[p.axis[pair] * rows + row] : pos0;
      const float turn2 = __ll2float_rn(static_cast<long long>(static_cast<uint64_t>(pos) * p.turns[pair])) * 0x1p-63f;
      float sn, cs;
      sincospif(turn2, &sn, &cs);
      rt.c[i] = cs;
      rt.s[i] = first ? -sign * sn : sign * sn;
    }
  }
}

// All 32 lanes call it (shuffles).
__device__ __forceinline__ void rotate(const Rotation& rt, float (&x)[8]) {
  float y[8];
  if (rt.inter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * rt.c[i] + x[i ^ 1] * rt.s[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * rt.c[i] + __shfl_sync(0xffffffffu, x[i], rt.src) * rt.s[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = y[i];
}

// Work unit u: row u / splits, head groups [g0, g1) of it.
struct Unit {
  int64_t row, b, r;
  int g0, g1;
  __device__ __forceinline__ Unit(const NormRopeParams& p, int64_t u, int splits, int groups) {
    row = u / splits;
    const int sp = static_cast<int>(u - row * splits);
    const int per = (groups + splits - 1) / splits;
    g0 = sp * per;
    g1 = min(groups, g0 + per);
    b = row / p.q_len;
    r = row - b * p.q_len;
  }
};

template <typename E, int D, bool kNorm>
__global__ void __launch_bounds__(kThreads)
    norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p, int splits, int64_t units) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, U = 4;
  const int lane = lane_id(), l = lane % LPH, sub = lane / LPH;
  const int heads = p.Hq + p.Hkv + (p.v_in != nullptr ? p.Hkv : 0);
  const int groups = (heads + HPW - 1) / HPW;
  float gq[8], gk[8];
  if constexpr (kNorm) {
    load8(static_cast<const E*>(p.gamma_q) + 8 * l, gq);
    load8(static_cast<const E*>(p.gamma_k) + 8 * l, gk);
  }
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp_id(); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Unit un(p, u, splits, groups);
    const E* xq = static_cast<const E*>(p.q_in) + un.row * p.q_stride + 8 * l;
    const E* xk = static_cast<const E*>(p.k_in) + un.row * p.k_stride + 8 * l;
    const E* xv = static_cast<const E*>(p.v_in) + un.row * p.v_stride + 8 * l;
    const int64_t cache_row = (un.b * p.T + p.q_start + un.r) * p.Hkv;
    E* yq = static_cast<E*>(p.q) + un.row * p.Hq * D + 8 * l;
    E* yk = static_cast<E*>(p.k_cache) + cache_row * D + 8 * l;
    E* yv = static_cast<E*>(p.v_cache) + cache_row * D + 8 * l;
    Rotation rt;
    bool have_rt = false;
    for (int g = un.g0; g < un.g1; g += U) {
      float x[U][8];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = (g + j) * HPW + sub;
        if (g + j < un.g1 && h < heads)
          load8(h < p.Hq ? xq + h * D : h < p.Hq + p.Hkv ? xk + (h - p.Hq) * D : xv + (h - p.Hq - p.Hkv) * D, x[j]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
      }
      if (!have_rt) {     // under the first loads' latency
        set_rotation<LPH>(rt, p, l, lane, un.row, p.q_start + un.r, 1.f);
        have_rt = true;
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = (g + j) * HPW + sub;
        if (g + j >= un.g1) break;               // warp-uniform
        float y[8];
        float r = 1.f;
        if constexpr (kNorm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += x[j][i] * x[j][i];
          r = 1.f / sqrtf(head_sum<LPH>(ss) * (1.f / D) + p.eps);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = x[j][i];
          if constexpr (kNorm) y[i] = y[i] * r * (h < p.Hq ? gq[i] : gk[i]);
        }
        if (p.rot_dim > 0) rotate(rt, y);
        if (h < p.Hq)
          store8(yq + h * D, y);
        else if (h < p.Hq + p.Hkv)
          store8(yk + (h - p.Hq) * D, y);
        else if (h < heads)
          store8(yv + (h - p.Hq - p.Hkv) * D, x[j]);
      }
    }
  }
}

template <typename E, int D, bool kNorm>
__global__ void __launch_bounds__(kThreads)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, int splits, int64_t units) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, U = 2;
  const int lane = lane_id(), l = lane % LPH, sub = lane / LPH;
  const int heads = p.Hq + p.Hkv + (p.dv_in != nullptr ? p.Hkv : 0);
  const int groups = (heads + HPW - 1) / HPW;
  float gq[8], gk[8], sq[8] = {}, sk[8] = {};
  if constexpr (kNorm) {
    load8(static_cast<const E*>(p.gamma_q) + 8 * l, gq);
    load8(static_cast<const E*>(p.gamma_k) + 8 * l, gk);
  }
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp_id(); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Unit un(p, u, splits, groups);
    const int64_t cache_row = (un.b * p.T + p.q_start + un.r) * p.Hkv;
    const E* xq = static_cast<const E*>(p.q_in) + un.row * p.q_stride + 8 * l;
    const E* xk = static_cast<const E*>(p.k_in) + un.row * p.k_stride + 8 * l;
    const float* gyq = p.dq + un.row * p.Hq * D + 8 * l;
    const float* gyk = p.dk + cache_row * D + 8 * l;
    const float* gyv = p.dv + cache_row * D + 8 * l;
    E* oq = static_cast<E*>(p.dq_in) + un.row * p.dq_stride + 8 * l;
    E* ok = static_cast<E*>(p.dk_in) + un.row * p.dk_stride + 8 * l;
    E* ov = static_cast<E*>(p.dv_in) + un.row * p.dv_stride + 8 * l;
    Rotation rt;
    bool have_rt = false;
    for (int g = un.g0; g < un.g1; g += U) {
      float x[U][8], dy[U][8];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = (g + j) * HPW + sub;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = dy[j][i] = 0.f;
        if (g + j < un.g1 && h < heads) {
          load8(h < p.Hq ? gyq + h * D : h < p.Hq + p.Hkv ? gyk + (h - p.Hq) * D : gyv + (h - p.Hq - p.Hkv) * D,
                dy[j]);
          if (kNorm && h < p.Hq + p.Hkv) load8(h < p.Hq ? xq + h * D : xk + (h - p.Hq) * D, x[j]);
        }
      }
      if (!have_rt) {
        set_rotation<LPH>(rt, p, l, lane, un.row, p.q_start + un.r, -1.f);
        have_rt = true;
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = (g + j) * HPW + sub;
        if (g + j >= un.g1) break;
        float dn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) dn[i] = dy[j][i];
        if (p.rot_dim > 0) rotate(rt, dn);
        if constexpr (kNorm) {
          float ss = 0.f, dot = 0.f;
          const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
          float gd[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            gd[i] = dn[i] * (is_q ? gq[i] : gk[i]);
            ss += x[j][i] * x[j][i];
            dot += gd[i] * x[j][i];
          }
          const float r = 1.f / sqrtf(head_sum<LPH>(ss) * (1.f / D) + p.eps);
          const float m = head_sum<LPH>(dot) * r * (1.f / D);     // mean(gamma dn xhat)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xh = x[j][i] * r;
            const float w = dn[i] * xh;
            if (is_q) sq[i] += w;
            if (is_k) sk[i] += w;
            dn[i] = r * (gd[i] - xh * m);
          }
        }
        if (h < p.Hq)
          store8(oq + h * D, dn);
        else if (h < p.Hq + p.Hkv)
          store8(ok + (h - p.Hq) * D, dn);
        else if (h < heads)
          store8(ov + (h - p.Hq - p.Hkv) * D, dy[j]);
      }
    }
  }
  if constexpr (kNorm) {
    // the block's share of dgamma, in a fixed order: heads of a warp, then warps
    __shared__ float part[kWarps][2][D];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = LPH; o < 32; o <<= 1) {
        sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
        sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], o);
      }
      if (sub == 0) {
        part[warp_id()][0][8 * l + i] = sq[i];
        part[warp_id()][1][8 * l + i] = sk[i];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += part[w][e / D][e % D];
      p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + e] = t;
    }
  }
}

// dgamma += the blocks' partial sums, in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024)
    norm_rope_dgamma_kernel(const float* __restrict__ partial, int blocks, float* dgamma_q, float* dgamma_k) {
  constexpr int kParts = 1024 / (2 * D);
  __shared__ float part[kParts][2 * D];
  const int e = threadIdx.x % (2 * D), w = threadIdx.x / (2 * D);
  float t = 0.f;
#pragma unroll 8
  for (int b = w; b < blocks; b += kParts) t += partial[static_cast<int64_t>(b) * 2 * D + e];
  part[w][e] = t;
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 1; i < kParts; ++i) t += part[i][e];
    float* dst = e < D ? dgamma_q + e : dgamma_k + (e - D);
    *dst += t;
  }
}

constexpr int kFillWarps = 152 * 32;      // warps that keep every SM's load queues busy
constexpr int kBwdBlocks = 152 * 2;

// Shares of a row's heads: rows alone fill the GPU, or the heads are dealt to
// enough warps that they do, down to one batch of loads per warp.
int splits_for(int64_t rows, int groups, int batch) {
  const int64_t want = (kFillWarps + rows - 1) / rows;
  const int most = (groups + batch - 1) / batch;
  return static_cast<int>(want < 1 ? 1 : want > most ? most : want);
}

template <typename E, int D>
cudaError_t fwd_typed(const NormRopeParams& p, cudaStream_t s) {
  const int hpw = 32 / (D / 8);
  const int64_t rows = static_cast<int64_t>(p.B) * p.q_len;
  const int heads = p.Hq + p.Hkv + (p.v_in != nullptr ? p.Hkv : 0);
  const int splits = splits_for(rows, (heads + hpw - 1) / hpw, 4);
  const int64_t units = rows * splits;
  const int64_t blocks = (units + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30));
  if (p.gamma_q != nullptr)
    norm_rope_fwd_kernel<E, D, true><<<grid, kThreads, 0, s>>>(p, splits, units);
  else
    norm_rope_fwd_kernel<E, D, false><<<grid, kThreads, 0, s>>>(p, splits, units);
  return cudaGetLastError();
}

template <typename E, int D>
cudaError_t bwd_typed(const NormRopeParams& p, cudaStream_t s) {
  const int hpw = 32 / (D / 8);
  const int64_t rows = static_cast<int64_t>(p.B) * p.q_len;
  const int heads = p.Hq + p.Hkv + (p.dv_in != nullptr ? p.Hkv : 0);
  const int splits = splits_for(rows, (heads + hpw - 1) / hpw, 2);
  const int64_t units = rows * splits;
  const int64_t blocks = (units + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(blocks < kBwdBlocks ? blocks : kBwdBlocks);
  if (p.gamma_q == nullptr) {
    norm_rope_bwd_kernel<E, D, false><<<grid, kThreads, 0, s>>>(p, splits, units);
    return cudaGetLastError();
  }
  norm_rope_bwd_kernel<E, D, true><<<grid, kThreads, 0, s>>>(p, splits, units);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_rope_dgamma_kernel<D><<<1, 1024, 0, s>>>(p.partial, grid, p.dgamma_q, p.dgamma_k);
  return cudaGetLastError();
}

}  // namespace

int norm_rope_bwd_blocks() { return kBwdBlocks; }

cudaError_t launch_norm_rope_fwd(const NormRopeParams& p, int d, bool bf16, cudaStream_t s) {
  if (bf16) return d == 64 ? fwd_typed<__nv_bfloat16, 64>(p, s) : fwd_typed<__nv_bfloat16, 128>(p, s);
  return d == 64 ? fwd_typed<float, 64>(p, s) : fwd_typed<float, 128>(p, s);
}

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, int d, bool bf16, cudaStream_t s) {
  if (bf16) return d == 64 ? bwd_typed<__nv_bfloat16, 64>(p, s) : bwd_typed<__nv_bfloat16, 128>(p, s);
  return d == 64 ? bwd_typed<float, 64>(p, s) : bwd_typed<float, 128>(p, s);
}

}  // namespace seqattn
