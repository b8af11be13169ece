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
// Heads are dealt in groups that fill a warp: eight elements a lane, d / 8 lanes
// a head, 32 / (d / 8) heads a group.  The (row, group) pairs of the call form
// one sequence, and every warp takes an equal stretch of it, so a single
// token's heads spread over the SMs and thousands of rows load them evenly by
// the same rule.  Within a row a lane's cosines and sines belong to its
// element indices: each lane computes those of two pairs (rot / 2 <= 64), and
// all lanes collect theirs by shuffles.  The partner of a half-split pair sits
// rot / 16 lanes away (its raw words are shuffled), that of an interleaved
// pair in the same lane.  Arithmetic runs on paired float32 instructions.
// Bound by HBM: every element is read and written once.
#include <cuda_bf16.h>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace seqattn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Eight consecutive elements as loaded: four words of bf16 pairs or eight of float32.
template <typename E>
struct Raw {
  static constexpr int kWords = 2 * sizeof(E);
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const E* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    if constexpr (sizeof(E) == 4) {
      const uint4 b = *reinterpret_cast<const uint4*>(p + 4);
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void store(E* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (sizeof(E) == 4) *reinterpret_cast<uint4*>(p + 4) = make_uint4(w[4], w[5], w[6], w[7]);
  }
  // as four float32 pairs
  __device__ __forceinline__ void unpack(uint64_t (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 2)
        f[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      else
        f[i] = f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
  }
  __device__ __forceinline__ void pack(const uint64_t (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2_unpack(f[i], a, b);
      if constexpr (sizeof(E) == 2) {
        w[i] = pack_bf16x2(a, b);
      } else {
        w[2 * i] = __float_as_uint(a);
        w[2 * i + 1] = __float_as_uint(b);
      }
    }
  }
  __device__ __forceinline__ Raw shuffled(int src) const {
    Raw r;
#pragma unroll
    for (int i = 0; i < kWords; ++i) r.w[i] = __shfl_sync(0xffffffffu, w[i], src);
    return r;
  }
};

__device__ __forceinline__ float f2_sum(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}
__device__ __forceinline__ uint64_t f2_swap(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return f2_pack(b, a);
}

// Sum over the LPH lanes of a head (every lane gets it; same order everywhere).
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What a lane keeps about the rotation for the whole call.
template <bool kInter>
struct LaneRotation {
  bool rotated;      // its elements lie below rot_dim
  int src;           // lane with the partners of its elements (half-split)
  int angle_src;     // first of the lanes that compute its angles
  float sign;        // of the sine in y = x cos + partner sin (first element of a pair)

  // `l`: lane within the head; `direction`: +1 forward, -1 backward
  __device__ __forceinline__ LaneRotation(const NormRopeParams& p, int l, int lane, float direction) {
    const int half = p.rot_dim / 2, e0 = 8 * l;
    rotated = e0 < p.rot_dim;
    const bool first = kInter || e0 < half;
    sign = first ? -direction : direction;
    src = !rotated || kInter ? lane : first ? lane + half / 8 : lane - half / 8;
    // pairs of this lane start at e0 / 2 (interleaved) or e0 modulo half
    angle_src = !rotated ? 0 : kInter ? e0 / 4 : (first ? e0 : e0 - half) / 2;
  }
};

// cos and sin of pairs 2 lane and 2 lane + 1 at this row (lanes past rot / 4
// compute something that no lane reads).
struct RowAngles {
  float c[2], s[2];
  __device__ __forceinline__ RowAngles(const NormRopeParams& p, int64_t row, int64_t pos0) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.q_len;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pair = 2 * lane_id() + i;
      const int64_t pos =
          p.positions != nullptr ? p.positions[(2 * pair < p.rot_dim ? p.axis[pair] : 0) * rows + row] : pos0;
      const float half_turns =
          __ll2float_rn(static_cast<long long>(static_cast<uint64_t>(pos) * p.turns[pair])) * 0x1p-63f;
      sincospif(half_turns, &s[i], &c[i]);
    }
  }
};

// The rotation of a lane's eight elements as float32 pairs:
// y = x c + partner(x) s, elementwise.  All 32 lanes call it (shuffles).
template <bool kInter>
__device__ __forceinline__ void spread(const LaneRotation<kInter>& lr, const RowAngles& a, uint64_t (&c)[4],
                                       uint64_t (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInter) {   // pair i of the lane: elements 2i, 2i + 1
      const int from = lr.angle_src + (i >> 1);
      const float cs = __shfl_sync(0xffffffffu, a.c[i & 1], from), sn = __shfl_sync(0xffffffffu, a.s[i & 1], from);
      c[i] = f2_pack(cs, cs);
      s[i] = f2_pack(lr.sign * sn, -lr.sign * sn);
    } else {                  // elements 2i, 2i + 1 belong to pairs 2i, 2i + 1 of the lane
      const int from = lr.angle_src + i;
      const float c0 = __shfl_sync(0xffffffffu, a.c[0], from), c1 = __shfl_sync(0xffffffffu, a.c[1], from);
      const float s0 = __shfl_sync(0xffffffffu, a.s[0], from), s1 = __shfl_sync(0xffffffffu, a.s[1], from);
      c[i] = f2_pack(c0, c1);
      s[i] = f2_pack(lr.sign * s0, lr.sign * s1);
    }
    if (!lr.rotated) {
      c[i] = f2_pack(1.f, 1.f);
      s[i] = f2_pack(0.f, 0.f);
    }
  }
}

// The groups of a row: query heads, then key heads, then value heads.
struct Groups {
  int q, k, v, all;
  __device__ __forceinline__ Groups(const NormRopeParams& p, int hpw, bool values) {
    q = (p.Hq + hpw - 1) / hpw;
    k = (p.Hkv + hpw - 1) / hpw;
    v = values ? k : 0;
    all = q + k + v;
  }
};

// This warp's stretch [begin, end) of the rows * groups sequence.
__device__ __forceinline__ void stretch(int64_t total, int64_t* begin, int64_t* end) {
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp_id();
  const int64_t each = total / warps, rest = total - each * warps;
  *begin = w * each + min(w, rest);
  *end = *begin + each + (w < rest ? 1 : 0);
}

// A place in the sequence: row, its row r within the batch entry, its first
// cached element, group g; moving to the next row divides nothing.
struct Place {
  int64_t row, cache;
  int r, g;
  __device__ __forceinline__ Place(const NormRopeParams& p, const Groups& gr, int64_t at, int d) {
    row = at / gr.all;
    g = static_cast<int>(at - row * gr.all);
    const int64_t b = row / p.q_len;
    r = static_cast<int>(row - b * p.q_len);
    cache = (b * p.T + p.q_start + r) * p.Hkv * d;
  }
  __device__ __forceinline__ void next_row(const NormRopeParams& p, int d) {
    g = 0;
    ++row;
    cache += p.Hkv * d;
    if (++r == p.q_len) {
      r = 0;
      cache += (p.T - p.q_len) * p.Hkv * d;
    }
  }
};

// Norm and rotation of the groups [g0, g1) of one kind (queries or keys) of a row.
template <typename E, int D, bool kNorm, bool kInter, int U>
__device__ __forceinline__ void fwd_heads(const NormRopeParams& p, const LaneRotation<kInter>& lr, const RowAngles& ang,
                                          const E* src, E* dst, const E* gamma, int heads, int g0, int g1) {
  constexpr int LPH = D / 8, HPW = 32 / LPH;
  const int lane = lane_id(), l = lane % LPH, sub = lane / LPH;
  src += sub * D + 8 * l;
  dst += sub * D + 8 * l;
  uint64_t c[4], s[4];
  bool ready = false;
  // the next U groups are loaded before the present ones are worked on
  Raw<E> next[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (g0 + j < g1 && (g0 + j) * HPW + sub < heads) next[j].load(src + (g0 + j) * (HPW * D));
    else next[j].zero();
  }
  for (int g = g0; g < g1; g += U) {
    Raw<E> x[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      x[j] = next[j];
      if (g + U + j < g1 && (g + U + j) * HPW + sub < heads) next[j].load(src + (g + U + j) * (HPW * D));
      else next[j].zero();
    }
    if (!ready) {            // under the first loads' latency
      ready = true;
      spread(lr, ang, c, s);
      if constexpr (kNorm) {
        // gamma goes into the coefficients: y = r (x gamma c + partner(x gamma) s)
        Raw<E> gm, gp;
        gm.load(gamma + 8 * l);
        gp = kInter ? gm : gm.shuffled(lr.src);
        uint64_t g2[4], gp2[4];
        gm.unpack(g2);
        gp.unpack(gp2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[i] = f2_mul(c[i], g2[i]);
          s[i] = f2_mul(s[i], kInter ? f2_swap(gp2[i]) : gp2[i]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (g + j >= g1) break;                    // warp-uniform
      uint64_t f[4], y[4];
      x[j].unpack(f);
      if constexpr (kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = f2_fma(f2_swap(f[i]), s[i], f2_mul(f[i], c[i]));
      } else {
        x[j].shuffled(lr.src).unpack(y);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = f2_fma(y[i], s[i], f2_mul(f[i], c[i]));
      }
      if constexpr (kNorm) {
        uint64_t ss = f2_mul(f[0], f[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = f2_fma(f[i], f[i], ss);
        const float r = rsqrtf(head_sum<LPH>(f2_sum(ss)) * (1.f / D) + p.eps);
        const uint64_t r2 = f2_pack(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = f2_mul(y[i], r2);
      }
      x[j].pack(y);
      if ((g + j) * HPW + sub < heads) x[j].store(dst + (g + j) * (HPW * D));
    }
  }
}

constexpr int kFwdBlocksPerSm = 2;

template <typename E, int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kThreads, kFwdBlocksPerSm)
    norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, U = 4;
  const int lane = lane_id(), l = lane % LPH, sub = lane / LPH;
  const Groups gr(p, HPW, p.v_in != nullptr);
  const LaneRotation<kInter> lr(p, l, lane, 1.f);
  int64_t at, end;
  grid_launch_dependents();
  grid_wait();
  stretch(static_cast<int64_t>(p.B) * p.q_len * gr.all, &at, &end);
  for (Place w(p, gr, at, D); at < end; w.next_row(p, D)) {
    const int g0 = w.g, g1 = static_cast<int>(min(static_cast<int64_t>(gr.all), g0 + (end - at)));
    at += g1 - g0;
    const int64_t row = w.row, cache = w.cache;
    const RowAngles ang(p, row, p.q_start + w.r);
    if (g0 < gr.q)
      fwd_heads<E, D, kNorm, kInter, U>(p, lr, ang, static_cast<const E*>(p.q_in) + row * p.q_stride,
                                static_cast<E*>(p.q) + row * p.Hq * D, static_cast<const E*>(p.gamma_q), p.Hq, g0,
                                min(g1, gr.q));
    if (g1 > gr.q && g0 < gr.q + gr.k)
      fwd_heads<E, D, kNorm, kInter, U>(p, lr, ang, static_cast<const E*>(p.k_in) + row * p.k_stride,
                                static_cast<E*>(p.k_cache) + cache, static_cast<const E*>(p.gamma_k), p.Hkv,
                                max(g0 - gr.q, 0), min(g1 - gr.q, gr.k));
    for (int g = max(g0 - gr.q - gr.k, 0); g < g1 - gr.q - gr.k; g += U) {      // values: copied as they are
      const E* src = static_cast<const E*>(p.v_in) + row * p.v_stride + sub * D + 8 * l;
      E* dst = static_cast<E*>(p.v_cache) + cache + sub * D + 8 * l;
      Raw<E> x[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (g + j < g1 - gr.q - gr.k && (g + j) * HPW + sub < p.Hkv) x[j].load(src + (g + j) * (HPW * D));
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (g + j < g1 - gr.q - gr.k && (g + j) * HPW + sub < p.Hkv) x[j].store(dst + (g + j) * (HPW * D));
    }
  }
}

// Backward of the groups [g0, g1) of one kind of a row; `acc` gathers this
// lane's share of dgamma.
template <typename E, int D, bool kNorm, bool kInter, int U>
__device__ __forceinline__ void bwd_heads(const NormRopeParams& p, const LaneRotation<kInter>& lr, const RowAngles& ang,
                                          const E* x_src, const float* dy_src, E* dst, const E* gamma, int heads,
                                          int g0, int g1, uint64_t (&acc)[4]) {
  constexpr int LPH = D / 8, HPW = 32 / LPH;
  const int lane = lane_id(), l = lane % LPH, sub = lane / LPH;
  const int64_t e0 = sub * D + 8 * l;
  uint64_t c[4], s[4];
  Raw<E> gamma_raw;
  bool ready = false;
  for (int g = g0; g < g1; g += U) {
    Raw<E> x[U];
    Raw<float> dy[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      dy[j].zero();
      x[j].zero();
      if (g + j < g1 && (g + j) * HPW + sub < heads) {
        dy[j].load(dy_src + e0 + (g + j) * (HPW * D));
        if constexpr (kNorm) x[j].load(x_src + e0 + (g + j) * (HPW * D));
      }
    }
    if (!ready) {
      ready = true;
      spread(lr, ang, c, s);
      if constexpr (kNorm) gamma_raw.load(gamma + 8 * l);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (g + j >= g1) break;                    // warp-uniform
      uint64_t d[4], dn[4];
      dy[j].unpack(d);
      if constexpr (kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dn[i] = f2_fma(f2_swap(d[i]), s[i], f2_mul(d[i], c[i]));
      } else {
        dy[j].shuffled(lr.src).unpack(dn);
#pragma unroll
        for (int i = 0; i < 4; ++i) dn[i] = f2_fma(dn[i], s[i], f2_mul(d[i], c[i]));
      }
      if constexpr (kNorm) {
        uint64_t f[4], gd[4];
        x[j].unpack(f);
        gamma_raw.unpack(gd);
#pragma unroll
        for (int i = 0; i < 4; ++i) gd[i] = f2_mul(gd[i], dn[i]);
        uint64_t ss = f2_mul(f[0], f[0]), dot = f2_mul(gd[0], f[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          ss = f2_fma(f[i], f[i], ss);
          dot = f2_fma(gd[i], f[i], dot);
        }
        const float r = rsqrtf(head_sum<LPH>(f2_sum(ss)) * (1.f / D) + p.eps);
        const float m = head_sum<LPH>(f2_sum(dot)) * r * (1.f / D);     // mean(gamma dn xhat)
        const uint64_t r2 = f2_pack(r, r), mr2 = f2_pack(-m * r, -m * r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t xh = f2_mul(f[i], r2);
          acc[i] = f2_fma(dn[i], xh, acc[i]);
          dn[i] = f2_fma(xh, mr2, f2_mul(gd[i], r2));
        }
      }
      Raw<E> out;
      out.pack(dn);
      if ((g + j) * HPW + sub < heads) out.store(dst + e0 + (g + j) * (HPW * D));
    }
  }
}

// Blocks per SM and groups in flight per warp, timed together: forward (4096
// rows, 64 + 8 + 8 heads of 128, bf16) 31.5 us with two blocks and 4 + 4
// groups, 34.4 without the loads ahead, 36 with 2 + 2, 37 with the next row
// prefetched into L2; backward (2048 rows, 32 + 8 + 8 heads, dgamma included)
// 25.2 us with one block and 4 groups, 28.2 with two blocks of 2, 26.2 with 6.
// With the groups ahead in a shared-memory ring (cp.async) the forward took
// 29.5 and the backward 27: even with its arithmetic and stores left out the
// backward's 63 MB of reads took 21 us, so neither more bytes in flight nor
// fewer instructions move it.
constexpr int kBwdBlocksPerSm = 1;

template <typename E, int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, U = 4;
  const int lane = lane_id(), l = lane % LPH, sub = lane / LPH;
  const Groups gr(p, HPW, p.dv_in != nullptr);
  const LaneRotation<kInter> lr(p, l, lane, -1.f);
  uint64_t sq[4] = {}, sk[4] = {};               // float32 pairs of zeros
  int64_t at, end;
  grid_launch_dependents();
  grid_wait();
  stretch(static_cast<int64_t>(p.B) * p.q_len * gr.all, &at, &end);
  for (Place w(p, gr, at, D); at < end; w.next_row(p, D)) {
    const int g0 = w.g, g1 = static_cast<int>(min(static_cast<int64_t>(gr.all), g0 + (end - at)));
    at += g1 - g0;
    const int64_t row = w.row, cache = w.cache;
    const RowAngles ang(p, row, p.q_start + w.r);
    if (g0 < gr.q)
      bwd_heads<E, D, kNorm, kInter, U>(p, lr, ang, static_cast<const E*>(p.q_in) + row * p.q_stride, p.dq + row * p.Hq * D,
                                static_cast<E*>(p.dq_in) + row * p.dq_stride, static_cast<const E*>(p.gamma_q), p.Hq,
                                g0, min(g1, gr.q), sq);
    if (g1 > gr.q && g0 < gr.q + gr.k)
      bwd_heads<E, D, kNorm, kInter, U>(p, lr, ang, static_cast<const E*>(p.k_in) + row * p.k_stride, p.dk + cache,
                                static_cast<E*>(p.dk_in) + row * p.dk_stride, static_cast<const E*>(p.gamma_k), p.Hkv,
                                max(g0 - gr.q, 0), min(g1 - gr.q, gr.k), sk);
    for (int g = max(g0 - gr.q - gr.k, 0); g < g1 - gr.q - gr.k; g += U) {      // values: rounded
      const float* src = p.dv + cache + sub * D + 8 * l;
      E* dst = static_cast<E*>(p.dv_in) + row * p.dv_stride + sub * D + 8 * l;
      Raw<float> x[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (g + j < g1 - gr.q - gr.k && (g + j) * HPW + sub < p.Hkv) x[j].load(src + (g + j) * (HPW * D));
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (g + j < g1 - gr.q - gr.k && (g + j) * HPW + sub < p.Hkv) {
          uint64_t f[4];
          Raw<E> out;
          x[j].unpack(f);
          out.pack(f);
          out.store(dst + (g + j) * (HPW * D));
        }
    }
  }
  if constexpr (kNorm) {
    // the block's share of dgamma, in a fixed order: heads of a warp, then warps
    __shared__ float part[kWarps][2][D];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[2];
        f2_unpack(kind == 0 ? sq[i] : sk[i], v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int o = LPH; o < 32; o <<= 1) v[h] += __shfl_xor_sync(0xffffffffu, v[h], o);
          if (sub == 0) part[warp_id()][kind][8 * l + 2 * i + h] = v[h];
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

// dgamma += the blocks' partial sums, in a fixed order.  A CTA owns 32 of the
// 2 d sums: warp w adds rows w, w + 32, ... of the partials, then warp 0 the
// 32 warps' sums.
template <int D>
__global__ void __launch_bounds__(1024)
    norm_rope_dgamma_kernel(const float* __restrict__ partial, int blocks, float* dgamma_q, float* dgamma_k) {
  __shared__ float part[32][32];
  const int lane = lane_id(), w = warp_id();
  const int e = blockIdx.x * 32 + lane;
  // launched while the backward still runs: wait until it has finished and its
  // partial sums are visible
  grid_wait();
  float t = 0.f;
#pragma unroll 4
  for (int b = w; b < blocks; b += 32) t += partial[static_cast<int64_t>(b) * 2 * D + e];
  part[w][lane] = t;
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) t += part[i][lane];
    float* dst = e < D ? dgamma_q + e : dgamma_k + (e - D);
    *dst += t;
  }
}

// One wave of blocks: as many as the registers let run at once, fewer when
// there is not a group for every warp.
constexpr int kSms = 152;
constexpr int kBwdBlocks = kSms * kBwdBlocksPerSm;

unsigned grid_for(const NormRopeParams& p, int hpw, bool values, int most) {
  const int groups = (p.Hq + hpw - 1) / hpw + (values ? 2 : 1) * ((p.Hkv + hpw - 1) / hpw);
  const int64_t blocks = (static_cast<int64_t>(p.B) * p.q_len * groups + kWarps - 1) / kWarps;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename E, int D>
cudaError_t fwd_typed(const NormRopeParams& p, cudaStream_t s) {
  const unsigned grid = grid_for(p, 32 / (D / 8), p.v_in != nullptr, kSms * kFwdBlocksPerSm);
  const bool norm = p.gamma_q != nullptr, inter = p.interleaved != 0;
  if (norm && inter) return launch_overlapped(norm_rope_fwd_kernel<E, D, true, true>, grid, kThreads, 0, 1, s, p);
  if (norm) return launch_overlapped(norm_rope_fwd_kernel<E, D, true, false>, grid, kThreads, 0, 1, s, p);
  if (inter) return launch_overlapped(norm_rope_fwd_kernel<E, D, false, true>, grid, kThreads, 0, 1, s, p);
  return launch_overlapped(norm_rope_fwd_kernel<E, D, false, false>, grid, kThreads, 0, 1, s, p);
}

template <typename E, int D>
cudaError_t bwd_typed(const NormRopeParams& p, cudaStream_t s) {
  const unsigned grid = grid_for(p, 32 / (D / 8), p.dv_in != nullptr, kBwdBlocks);
  const bool inter = p.interleaved != 0;
  if (p.gamma_q == nullptr) {
    if (inter) return launch_overlapped(norm_rope_bwd_kernel<E, D, false, true>, grid, kThreads, 0, 1, s, p);
    return launch_overlapped(norm_rope_bwd_kernel<E, D, false, false>, grid, kThreads, 0, 1, s, p);
  }
  const cudaError_t e =
      inter ? launch_overlapped(norm_rope_bwd_kernel<E, D, true, true>, grid, kThreads, 0, 1, s, p)
            : launch_overlapped(norm_rope_bwd_kernel<E, D, true, false>, grid, kThreads, 0, 1, s, p);
  if (e != cudaSuccess) return e;
  return launch_overlapped(norm_rope_dgamma_kernel<D>, 2 * D / 32, 1024, 0, 1, s,
                           static_cast<const float*>(p.partial), static_cast<int>(grid), p.dgamma_q, p.dgamma_k);
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
