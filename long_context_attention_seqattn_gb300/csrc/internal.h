// internal.h -- launch plumbing shared between the C-ABI front end and the
// kernel translation units of libseqattn.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace seqattn {

// Geometry of one chunk call, after validation.
struct ChunkGeom {
  int B, Hq, Hkv, G, d;
  int64_t T;         // cache rows
  int64_t q_start;   // absolute row of the chunk's first query
  int64_t q_len;     // rows in the chunk
  int64_t kv_begin;  // first visible key row (q_start - prefix_len)
  float scale;       // softmax scale
  long long wait_cycles;  // limit of every bounded device wait (SM cycles)
};

// ---- float32 exact path (SIMT FMA) ----------------------------------------
cudaError_t launch_fwd_f32(const ChunkGeom& g, const float* q, const float* k, const float* v,
                           float* o, float* lse, unsigned int* err, cudaStream_t s);
cudaError_t launch_bwd_f32(const ChunkGeom& g, const float* q, const float* k, const float* v,
                           const float* lse, const float* d_o, const float* delta, float* dq,
                           float* dk, float* dv, unsigned int* err, cudaStream_t s);

// ---- Delta = rowsum(dO o O) and the backward row statistics ---------------
// bf16 path: per 64-row query tile, -L log2(e) and Delta side by side in a
// padded [B, Hq, ceil(q_len / 64), 2, 64] float32 array (padding rows -inf, 0);
// also zeroes dq.
cudaError_t launch_bwd_stats_bf16(const ChunkGeom& g, const void* o, const void* d_o,
                                  const float* lse, float* stats, float* dq, cudaStream_t s);
cudaError_t launch_bwd_prep_f32(const ChunkGeom& g, const float* o, const float* d_o,
                                float* delta, cudaStream_t s);

// ---- zero fill of the float32 accumulators ---------------------------------
cudaError_t launch_zero_f32(float* a, float* b, int64_t n, cudaStream_t s);
// rows [r0, r1) of two [B, T, row_floats] float32 arrays times `scale` (0 stores zeros)
cudaError_t launch_scale_rows_f32(float* a, float* b, int B, int64_t T, int64_t r0, int64_t r1,
                                  int64_t row_floats, float scale, cudaStream_t s);

// ---- bf16 tensor-core path (TMA + tcgen05 + TMEM) -------------------------
// Tensor maps are built by the front end (make_map in seqattn_api.cu).
struct Bf16FwdMaps {
  CUtensorMap q, k, v;
};
struct Bf16BwdMaps {
  CUtensorMap q, k, v, d_o;
  CUtensorMap dk, dv;   // fp32 [B][rows < q_end][Hkv][d], box {32, 1, 128, 1}, 128-byte swizzle
};
cudaError_t launch_fwd_bf16(const ChunkGeom& g, const Bf16FwdMaps& maps, void* o, float* lse,
                            unsigned int* err, cudaStream_t s);
// `stats` as written by launch_bwd_stats_bf16.
cudaError_t launch_bwd_bf16(const ChunkGeom& g, const Bf16BwdMaps& maps, const float* stats,
                            float* dq, float* dk, float* dv, unsigned int* err, cudaStream_t s);

// ---- projection weight gradient (tcgen05, G rounded to bf16 in the kernel) -
// Rows (tokens) per pipeline stage: the height of the h and g boxes.
constexpr int kWgradStageRows = 64;
// h: bf16 [B, T, d_model], box {64 columns, kWgradStageRows rows, 1}, 128-byte swizzle;
// g: fp32 [B, T, n], box {128 columns, kWgradStageRows rows, 1}, no swizzle;
// dw: fp32 [1, d_model, n], box {128 columns, 32 rows, 1}, no swizzle (the
// target of the epilogue's reduce-adds).
struct WgradMaps {
  CUtensorMap h, g, dw;
};
cudaError_t launch_wgrad_bf16(const WgradMaps& maps, int32_t batch, int64_t row_begin, int64_t row_end,
                              int32_t d_model, int32_t n, unsigned int* err, long long wait_cycles,
                              cudaStream_t s);

// ---- linear layer: products with epilogues (tcgen05) ------------------------
enum : int { kLinearFwd = 0, kLinearDgrad = 1, kLinearWgrad = 2 };
enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };
// Contraction elements per pipeline stage.
constexpr int kLinearStageK = 64;
struct LinearMaps {
  CUtensorMap a, b;
  CUtensorMap out;             // wgrad: float32 result, box {32, 32}, 128-byte swizzle
};
// Rows of an operand box of a K-major operand: a tile's 128.  A result of
// fewer than 128 rows has its A in boxes of those rows, rounded up to the
// swizzle's 8: the tile's other rows hold whatever the ring holds, and only
// result rows that are never stored depend on them.
constexpr int linear_a_rows(int64_t m) { return m >= 128 ? 128 : static_cast<int>((m + 7) / 8 * 8); }
constexpr uint32_t linear_a_bytes(int64_t m) { return static_cast<uint32_t>(linear_a_rows(m) * kLinearStageK * 2); }
struct LinearParams {
  int m, n, k;                 // result rows and columns, contraction length
  int act;
  const __nv_bfloat16* bias;   // [n], forward
  const __nv_bfloat16* residual;
  __nv_bfloat16* z;            // pre-activation: written by the forward, read by dgrad
  void* out;                   // bf16 (forward, dgrad) or float32 accumulator (wgrad)
  int64_t ldr, ldz, ldo;       // row strides in elements
  // filled by plan_linear_bf16
  int pair_tiles, tile_n;      // tiles of the pair shape and their columns
  int pairs;                   // pairs that run at once
  int split_tiles, split;      // small tiles and the CTAs that share one: the
                               // whole result, or the quarters of what the pairs leave
  // filled by the launch: this kernel's tiles, and the pairs' first tile it quarters (-1: none)
  int tiles, tail_base;
  uint32_t a_bytes;            // bytes of one A tile's copies (split shape)
  int a_blocked, b_blocked;    // MN-major operand's map has its 64-column blocks as a dimension
  unsigned int* err;
  long long wait_cycles;
};
cudaError_t plan_linear_bf16(int mode, LinearParams& p);
cudaError_t launch_linear_bf16(int mode, const LinearMaps& maps, const LinearParams& p, cudaStream_t s);
// forward of at most kLinearGemvRows rows without the tensor cores
constexpr int kLinearGemvRows = 2;
cudaError_t launch_linear_gemv(const LinearParams& p, const void* x, int64_t ldx, const void* w, cudaStream_t s);
// dbias[j] += sum over rows of g[r, j] (bf16), in a fixed order
cudaError_t launch_colsum_bf16(const void* g, int64_t ldg, int rows, int n, float* dbias, cudaStream_t s);

// ---- head norm + rotary positions + cache write ------------------------------
struct NormRopeParams {
  int B, q_len, Hq, Hkv;
  int64_t T, q_start;
  // forward: x = q/k/v inputs, y = q chunk and caches; backward: see the kernel
  const void *q_in, *k_in, *v_in;      // element type, rows of `*_stride` elements
  int64_t q_stride, k_stride, v_stride;
  const void *gamma_q, *gamma_k;       // element type [d], or NULL
  float eps;
  const int64_t* positions;            // [axes, B, q_len], or NULL (q_start + row)
  void *q, *k_cache, *v_cache;         // forward outputs
  const float *dq, *dk, *dv;           // backward inputs
  void *dq_in, *dk_in, *dv_in;         // backward outputs, rows of `d*_stride` elements
  int64_t dq_stride, dk_stride, dv_stride;
  float* partial;                      // backward: [blocks, 2, d] partial dgamma
  float *dgamma_q, *dgamma_k;
  int rot_dim, axes, interleaved;      // rot_dim 0: no rotation
  uint64_t turns[64];                  // turns per position, in units of 2^-64
  uint8_t axis[64];
};
cudaError_t launch_norm_rope_fwd(const NormRopeParams& p, int d, bool bf16, cudaStream_t s);
// most blocks of the backward's grid, and so rows of `partial`
int norm_rope_bwd_blocks();
cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, int d, bool bf16, cudaStream_t s);

// ---- AdamW over many tensors ---------------------------------------------------
struct AdamwTensor {          // mirrors seqattn_adamw_tensor
  float* param;
  void* lowp;                 // bf16 copy of param, or NULL
  const void* grad;
  void *m, *v;                // float32, or e4m3 codes
  float *m_scale, *v_scale;   // 8-bit states: one scale per 256 elements
  int64_t n;
  float weight_decay;
  int32_t grad_bf16;
};
struct AdamwHyper {
  float lr, beta1, one_minus_beta1, beta2, one_minus_beta2, eps, grad_scale;
  float step_size, inv_root_bc2;   // lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
  double lrd, beta1d, beta2d;
  int64_t step;
  const float* lr_dev;             // device values that replace the host's, or NULL
  const float* grad_scale_dev;
  const int64_t* step_dev;
};
constexpr int kAdamwBlock = 256;   // elements per 8-bit scale
cudaError_t launch_adamw(const AdamwTensor* t, int count, int state_bits, const AdamwHyper& h, cudaStream_t s);

// ---- launches that may overlap their predecessor's end (kernels with grid_wait) ---
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                              cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace seqattn
