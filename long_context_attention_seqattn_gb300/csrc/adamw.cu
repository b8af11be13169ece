// adamw.cu -- one AdamW step over many tensors in one launch, with the moments
// in float32 or in 8 bits:
//   g = grad_scale * grad
//   m = b1 m + (1 - b1) g,   v = b2 v + ((1 - b2) g) g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// p is the float32 master weight; a bf16 copy for the next forward is written
// in the same pass.  Every operation is rounded to float32 by itself, in this
// order (no contraction), so the states do not depend on how the compiler fuses
// it: 8-bit codes in particular are reproducible.  Only the quotient of p's
// step is the fast one (2 ulp of a term that is a small part of p).
//
// 8-bit states: 256 consecutive elements share one float32 scale, max |x| / 448,
// and each is stored as the nearest e4m3 number of x / scale.  The second
// moment is stored as u = sqrt(v): its range in binades is half of v's, which
// e4m3 covers.  A u that would round to zero is stored as the smallest code
// instead: with u = 0 and an m that is not, the step would explode.  A block
// whose maximum is under 1e-30 stores zeros.
//
// Bound by HBM: 30 bytes a parameter (float32 states, float32 gradient, bf16
// copy), 18 with 8-bit states.  One warp owns a block of 256 elements, four
// consecutive ones a lane twice, so every access is a full 16-byte (float32),
// 8-byte (bf16) or 4-byte (e4m3) vector of consecutive lanes, and the block's
// maximum is a warp reduction.  The tensors' descriptors travel in the launch
// parameters: no device copy of the list, and a captured graph keeps its own.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace seqattn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int64_t kBlockElems = kWarps * kAdamwBlock;   // elements per CTA

template <int kCap>
struct AdamwList {
  AdamwTensor t[kCap];
  uint32_t first[kCap + 1];   // CTA index of each tensor's first block
  int count;
};

__device__ __forceinline__ void decode4(uint32_t codes, float scale, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes >> (16 * i))));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = __fmul_rn(v.x, scale);
    f[2 * i + 1] = __fmul_rn(v.y, scale);
  }
}

__device__ __forceinline__ uint32_t encode4(const float (&f)[4], float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fmul_rn(f[1], inv)), "f"(__fmul_rn(f[0], inv)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fmul_rn(f[3], inv)), "f"(__fmul_rn(f[2], inv)));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// kDev: scalars may come from the device.
template <bool k8, bool kDev, int kCap>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ AdamwList<kCap> list, const __grid_constant__ AdamwHyper h) {
  // ---- tensor of this CTA (the last one that starts at or before it)
  int lo = 0, hi = list.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (list.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamwTensor& t = list.t[lo];
  const int64_t block = static_cast<int64_t>(blockIdx.x - list.first[lo]) * kWarps + warp_id();   // 256-element block
  const int64_t e0 = block * kAdamwBlock;

  // ---- the step's scalars
  float lr = h.lr, step_size = h.step_size, inv_root = h.inv_root_bc2, gscale = h.grad_scale;
  if constexpr (kDev) {
    // one thread of the CTA raises the betas to the step (float64: 1 - beta^t cancels)
    __shared__ float sh_step_size, sh_inv_root;
    if (h.lr_dev != nullptr) lr = *h.lr_dev;
    if (h.grad_scale_dev != nullptr) gscale = __fmul_rn(gscale, *h.grad_scale_dev);
    if (threadIdx.x == 0) {
      const double n = static_cast<double>(h.step_dev != nullptr ? *h.step_dev : h.step);
      sh_step_size = static_cast<float>((h.lr_dev != nullptr ? static_cast<double>(lr) : h.lrd) / (1.0 - pow(h.beta1d, n)));
      sh_inv_root = __fdiv_rn(1.f, static_cast<float>(sqrt(1.0 - pow(h.beta2d, n))));
    }
    __syncthreads();
    step_size = sh_step_size;
    inv_root = sh_inv_root;
  }
  if (e0 >= t.n) return;                         // warp-uniform
  const float decay = __fsub_rn(1.f, __fmul_rn(lr, t.weight_decay));

  const int lane = lane_id();
  const bool whole = e0 + kAdamwBlock <= t.n;
  float p[2][4], g[2][4], m[2][4], v[2][4];
  float ms = 0.f, us = 0.f;
  if constexpr (k8) {
    ms = t.m_scale[block];
    us = t.v_scale[block];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t e = e0 + 128 * j + 4 * lane;
    if (whole) {
      const float4 pv = *reinterpret_cast<const float4*>(t.param + e);
      p[j][0] = pv.x, p[j][1] = pv.y, p[j][2] = pv.z, p[j][3] = pv.w;
      if (t.grad_bf16) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(t.grad) + e);
        g[j][0] = __uint_as_float(q.x << 16), g[j][1] = __uint_as_float(q.x & 0xffff0000u);
        g[j][2] = __uint_as_float(q.y << 16), g[j][3] = __uint_as_float(q.y & 0xffff0000u);
      } else {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(t.grad) + e);
        g[j][0] = q.x, g[j][1] = q.y, g[j][2] = q.z, g[j][3] = q.w;
      }
      if constexpr (k8) {
        decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + e), ms, m[j]);
        decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + e), us, v[j]);
      } else {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(t.m) + e);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(t.v) + e);
        m[j][0] = a.x, m[j][1] = a.y, m[j][2] = a.z, m[j][3] = a.w;
        v[j][0] = b.x, v[j][1] = b.y, v[j][2] = b.z, v[j][3] = b.w;
      }
    } else {
      // the tensor's last block: element by element, nothing past n is touched
      uint32_t cm = 0, cu = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = e + i < t.n;
        p[j][i] = in ? t.param[e + i] : 0.f;
        g[j][i] = !in ? 0.f
                  : t.grad_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[e + i])
                                : static_cast<const float*>(t.grad)[e + i];
        if constexpr (k8) {
          cm |= in ? static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[e + i]) << (8 * i) : 0u;
          cu |= in ? static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[e + i]) << (8 * i) : 0u;
        } else {
          m[j][i] = in ? static_cast<const float*>(t.m)[e + i] : 0.f;
          v[j][i] = in ? static_cast<const float*>(t.v)[e + i] : 0.f;
        }
      }
      if constexpr (k8) {
        decode4(cm, ms, m[j]);
        decode4(cu, us, v[j]);
      }
    }
  }
  float mtop = 0.f, utop = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gg = __fmul_rn(g[j][i], gscale);
      const float vv = k8 ? __fmul_rn(v[j][i], v[j][i]) : v[j][i];
      const float mm = __fadd_rn(__fmul_rn(h.beta1, m[j][i]), __fmul_rn(h.one_minus_beta1, gg));
      const float vn = __fadd_rn(__fmul_rn(h.beta2, vv), __fmul_rn(__fmul_rn(h.one_minus_beta2, gg), gg));
      const float root = __fsqrt_rn(vn);
      const float denom = __fadd_rn(__fmul_rn(root, inv_root), h.eps);
      p[j][i] = __fsub_rn(__fmul_rn(p[j][i], decay), __fmul_rn(step_size, __fdividef(mm, denom)));
      m[j][i] = mm;
      v[j][i] = k8 ? root : vn;
      if constexpr (k8) {
        mtop = fmaxf(mtop, fabsf(mm));
        utop = fmaxf(utop, root);
      }
    }
  float minv = 0.f, uinv = 0.f;
  if constexpr (k8) {
    mtop = warp_max(mtop);
    utop = warp_max(utop);
    if (mtop < 1e-30f) mtop = 0.f;
    if (utop < 1e-30f) utop = 0.f;
    minv = mtop > 0.f ? __fdiv_rn(448.f, mtop) : 0.f;
    uinv = utop > 0.f ? __fdiv_rn(448.f, utop) : 0.f;
    if (lane == 0) {
      t.m_scale[block] = __fmul_rn(mtop, 1.f / 448.f);
      t.v_scale[block] = __fmul_rn(utop, 1.f / 448.f);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t e = e0 + 128 * j + 4 * lane;
    uint32_t cm = 0, cu = 0;
    if constexpr (k8) {
      cm = encode4(m[j], minv);
      cu = encode4(v[j], uinv);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (((cu >> (8 * i)) & 0xffu) == 0u && v[j][i] > 0.f && utop > 0.f) cu |= 1u << (8 * i);
    }
    if (whole) {
      *reinterpret_cast<float4*>(t.param + e) = make_float4(p[j][0], p[j][1], p[j][2], p[j][3]);
      if (t.lowp != nullptr)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(t.lowp) + e) =
            make_uint2(pack_bf16x2(p[j][0], p[j][1]), pack_bf16x2(p[j][2], p[j][3]));
      if constexpr (k8) {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + e) = cm;
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + e) = cu;
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(t.m) + e) = make_float4(m[j][0], m[j][1], m[j][2], m[j][3]);
        *reinterpret_cast<float4*>(static_cast<float*>(t.v) + e) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= t.n) break;
        t.param[e + i] = p[j][i];
        if (t.lowp != nullptr) static_cast<__nv_bfloat16*>(t.lowp)[e + i] = __float2bfloat16_rn(p[j][i]);
        if constexpr (k8) {
          static_cast<uint8_t*>(t.m)[e + i] = static_cast<uint8_t>(cm >> (8 * i));
          static_cast<uint8_t*>(t.v)[e + i] = static_cast<uint8_t>(cu >> (8 * i));
        } else {
          static_cast<float*>(t.m)[e + i] = m[j][i];
          static_cast<float*>(t.v)[e + i] = v[j][i];
        }
      }
    }
  }
}

// Tensors of one launch: the large list is close to the 32764 bytes of launch
// parameters, the small one keeps a short list's launch short.
constexpr int kCapLarge = 384;
constexpr int kCapSmall = 32;

template <int kCap>
cudaError_t launch_list(const AdamwTensor* t, int count, int state_bits, const AdamwHyper& h, cudaStream_t s) {
  AdamwList<kCap> list;
  static_assert(sizeof(list) + sizeof(h) <= 32764, "launch parameters");
  list.count = count;
  uint64_t blocks = 0;
  for (int i = 0; i < count; ++i) {
    list.t[i] = t[i];
    list.first[i] = static_cast<uint32_t>(blocks);
    blocks += static_cast<uint64_t>((t[i].n + kBlockElems - 1) / kBlockElems);
  }
  if (blocks == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(blocks);
  const bool dev = h.lr_dev != nullptr || h.grad_scale_dev != nullptr || h.step_dev != nullptr;
  if (state_bits == 8) {
    if (dev) adamw_kernel<true, true, kCap><<<grid, kThreads, 0, s>>>(list, h);
    else adamw_kernel<true, false, kCap><<<grid, kThreads, 0, s>>>(list, h);
  } else {
    if (dev) adamw_kernel<false, true, kCap><<<grid, kThreads, 0, s>>>(list, h);
    else adamw_kernel<false, false, kCap><<<grid, kThreads, 0, s>>>(list, h);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamwTensor* t, int count, int state_bits, const AdamwHyper& h, cudaStream_t s) {
  int at = 0;
  while (at < count) {
    // as many tensors as one launch's list and grid can hold
    int take = 0;
    uint64_t blocks = 0;
    while (at + take < count && take < kCapLarge) {
      const uint64_t more = static_cast<uint64_t>((t[at + take].n + kBlockElems - 1) / kBlockElems);
      if (take > 0 && blocks + more > 0x7fffffffull) break;
      blocks += more;
      ++take;
    }
    const cudaError_t e = take <= kCapSmall ? launch_list<kCapSmall>(t + at, take, state_bits, h, s)
                                            : launch_list<kCapLarge>(t + at, take, state_bits, h, s);
    if (e != cudaSuccess) return e;
    at += take;
  }
  return cudaSuccess;
}

}  // namespace seqattn
