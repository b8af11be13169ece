// adamw.cu -- one AdamW step over many tensors in one launch, with the moments
// in float32 or in 8 bits:
//   g = grad_scale * grad
//   m = b1 m + (1 - b1) g,   v = b2 v + ((1 - b2) g) g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// p is the float32 master weight; a bf16 copy for the next forward is written
// in the same pass.  The operations of m, v and sqrt(v) are rounded to float32
// one by one, in this order, so the states, and the 8-bit codes in particular,
// do not depend on how the compiler fuses them (one code that falls to the
// other side of a border moves a value by a sixteenth).  In p's step products
// and sums may be fused and the quotient is the fast one: 2 ulp of a term that
// is a small part of p.
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

// Four e4m3 codes as float32 pairs times the scale.
__device__ __forceinline__ void decode4(uint32_t codes, uint64_t scale2, uint64_t (&f)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes >> (16 * i))));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[i] = f2_mul(f2_pack(v.x, v.y), scale2);
  }
}

__device__ __forceinline__ uint32_t encode4(const float (&f)[4]) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Largest of the warp's values, none of them negative or NaN: their bit
// patterns then order as the numbers do.
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// a + b of float32 pairs by single additions: a paired multiplication and a
// paired addition after it are fused into one rounding by the assembler, even
// with explicit rounding.
__device__ __forceinline__ uint64_t sum_rn(uint64_t a, uint64_t b) {
  float a0, a1, b0, b1;
  f2_unpack(a, a0, a1);
  f2_unpack(b, b0, b1);
  return f2_pack(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}

__device__ __forceinline__ uint64_t both(float v) { return f2_pack(v, v); }

// kDev: scalars may come from the device.
template <bool k8, bool kDev, int kCap>
__global__ void __launch_bounds__(kThreads, k8 ? 5 : 4)   // 8 bit: 130 us with 5 blocks an SM, 138 with 4
    adamw_kernel(const __grid_constant__ AdamwList<kCap> list, const __grid_constant__ AdamwHyper h) {
  grid_launch_dependents();
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

  grid_wait();
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
  uint64_t p[2][2], g[2][2], m[2][2], v[2][2];   // float32 pairs; v is u in the 8-bit form
  uint64_t ms = 0, us = 0;
  if constexpr (k8) {
    ms = both(t.m_scale[block]);
    us = both(t.v_scale[block]);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t e = e0 + 128 * j + 4 * lane;
    if (whole) {
      const float4 pv = *reinterpret_cast<const float4*>(t.param + e);
      p[j][0] = f2_pack(pv.x, pv.y), p[j][1] = f2_pack(pv.z, pv.w);
      if (t.grad_bf16) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(t.grad) + e);
        g[j][0] = f2_pack(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u));
        g[j][1] = f2_pack(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
      } else {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(t.grad) + e);
        g[j][0] = f2_pack(q.x, q.y), g[j][1] = f2_pack(q.z, q.w);
      }
      if constexpr (k8) {
        decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + e), ms, m[j]);
        decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + e), us, v[j]);
      } else {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(t.m) + e);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(t.v) + e);
        m[j][0] = f2_pack(a.x, a.y), m[j][1] = f2_pack(a.z, a.w);
        v[j][0] = f2_pack(b.x, b.y), v[j][1] = f2_pack(b.z, b.w);
      }
    } else {
      // the tensor's last block: element by element, nothing past n is touched
      uint32_t cm = 0, cu = 0;
      float pe[4], ge[4], me[4], ve[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = e + i < t.n;
        pe[i] = in ? t.param[e + i] : 0.f;
        ge[i] = !in ? 0.f
                : t.grad_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[e + i])
                              : static_cast<const float*>(t.grad)[e + i];
        if constexpr (k8) {
          cm |= in ? static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[e + i]) << (8 * i) : 0u;
          cu |= in ? static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[e + i]) << (8 * i) : 0u;
        } else {
          me[i] = in ? static_cast<const float*>(t.m)[e + i] : 0.f;
          ve[i] = in ? static_cast<const float*>(t.v)[e + i] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        p[j][i] = f2_pack(pe[2 * i], pe[2 * i + 1]);
        g[j][i] = f2_pack(ge[2 * i], ge[2 * i + 1]);
        if constexpr (!k8) {
          m[j][i] = f2_pack(me[2 * i], me[2 * i + 1]);
          v[j][i] = f2_pack(ve[2 * i], ve[2 * i + 1]);
        }
      }
      if constexpr (k8) {
        decode4(cm, ms, m[j]);
        decode4(cu, us, v[j]);
      }
    }
  }
  // ---- the step, paired instructions that round each product and sum
  const uint64_t gs2 = both(gscale), b1 = both(h.beta1), c1 = both(h.one_minus_beta1), b2 = both(h.beta2),
                 c2 = both(h.one_minus_beta2), ir2 = both(inv_root), eps2 = both(h.eps), decay2 = both(decay);
  float mtop = 0.f, utop = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t gg = f2_mul(g[j][i], gs2);
      const uint64_t vv = k8 ? f2_mul(v[j][i], v[j][i]) : v[j][i];
      const uint64_t mm = sum_rn(f2_mul(b1, m[j][i]), f2_mul(c1, gg));
      const uint64_t vn = sum_rn(f2_mul(b2, vv), f2_mul(f2_mul(c2, gg), gg));
      float ma, mb, va, vb, da, db;
      f2_unpack(mm, ma, mb);
      f2_unpack(vn, va, vb);
      const float ra = __fsqrt_rn(va), rb = __fsqrt_rn(vb);
      f2_unpack(f2_add(f2_mul(f2_pack(ra, rb), ir2), eps2), da, db);
      const uint64_t step = f2_pack(__fmul_rn(step_size, __fdividef(ma, da)), __fmul_rn(step_size, __fdividef(mb, db)));
      p[j][i] = f2_sub(f2_mul(p[j][i], decay2), step);
      m[j][i] = mm;
      v[j][i] = k8 ? f2_pack(ra, rb) : vn;
      if constexpr (k8) {
        mtop = fmaxf(mtop, fmaxf(fabsf(ma), fabsf(mb)));
        utop = fmaxf(utop, fmaxf(ra, rb));
      }
    }
  uint64_t minv = 0, uinv = 0;
  float least = 0.f;            // smallest code of a positive u
  if constexpr (k8) {
    mtop = warp_max(mtop);
    utop = warp_max(utop);
    if (mtop < 1e-30f) mtop = 0.f;
    if (utop < 1e-30f) utop = 0.f;
    minv = both(mtop > 0.f ? __fmul_rn(448.f, __frcp_rn(mtop)) : 0.f);
    uinv = both(utop > 0.f ? __fmul_rn(448.f, __frcp_rn(utop)) : 0.f);
    least = utop > 0.f ? 0x1p-9f : 0.f;
    if (lane == 0) {
      t.m_scale[block] = __fmul_rn(mtop, 1.f / 448.f);
      t.v_scale[block] = __fmul_rn(utop, 1.f / 448.f);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t e = e0 + 128 * j + 4 * lane;
    float pe[4], me[4], ve[4];
    uint32_t cm = 0, cu = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f2_unpack(p[j][i], pe[2 * i], pe[2 * i + 1]);
      f2_unpack(k8 ? f2_mul(m[j][i], minv) : m[j][i], me[2 * i], me[2 * i + 1]);
      f2_unpack(k8 ? f2_mul(v[j][i], uinv) : v[j][i], ve[2 * i], ve[2 * i + 1]);
      if constexpr (k8) {
        // above 2^-10 the nearest code is at least 2^-9 anyway
        float a, b;
        f2_unpack(v[j][i], a, b);
        ve[2 * i] = fmaxf(ve[2 * i], a > 0.f ? least : ve[2 * i]);
        ve[2 * i + 1] = fmaxf(ve[2 * i + 1], b > 0.f ? least : ve[2 * i + 1]);
      }
    }
    if constexpr (k8) {
      cm = encode4(me);
      cu = encode4(ve);
    }
    if (whole) {
      *reinterpret_cast<float4*>(t.param + e) = make_float4(pe[0], pe[1], pe[2], pe[3]);
      if (t.lowp != nullptr)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(t.lowp) + e) =
            make_uint2(pack_bf16x2(pe[0], pe[1]), pack_bf16x2(pe[2], pe[3]));
      if constexpr (k8) {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + e) = cm;
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + e) = cu;
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(t.m) + e) = make_float4(me[0], me[1], me[2], me[3]);
        *reinterpret_cast<float4*>(static_cast<float*>(t.v) + e) = make_float4(ve[0], ve[1], ve[2], ve[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (e + i >= t.n) break;
        t.param[e + i] = pe[i];
        if (t.lowp != nullptr) static_cast<__nv_bfloat16*>(t.lowp)[e + i] = __float2bfloat16_rn(pe[i]);
        if constexpr (k8) {
          static_cast<uint8_t*>(t.m)[e + i] = static_cast<uint8_t>(cm >> (8 * i));
          static_cast<uint8_t*>(t.v)[e + i] = static_cast<uint8_t>(cu >> (8 * i));
        } else {
          static_cast<float*>(t.m)[e + i] = me[i];
          static_cast<float*>(t.v)[e + i] = ve[i];
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
    if (dev) return launch_overlapped(adamw_kernel<true, true, kCap>, grid, kThreads, 0, 1, s, list, h);
    return launch_overlapped(adamw_kernel<true, false, kCap>, grid, kThreads, 0, 1, s, list, h);
  }
  if (dev) return launch_overlapped(adamw_kernel<false, true, kCap>, grid, kThreads, 0, 1, s, list, h);
  return launch_overlapped(adamw_kernel<false, false, kCap>, grid, kThreads, 0, 1, s, list, h);
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
