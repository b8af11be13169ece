// seqattn_api.cu -- the C ABI declared in include/seqattn.h: argument
// validation (before any launch), TMA tensor maps, the per-device error word,
// and dispatch to the float32 and bf16 kernel families, the accumulator row
// scaling, the projection weight gradient kernel, the linear layer's products,
// the head norm with rotary positions and the optimizer step.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <mutex>
#include <string>

#include "internal.h"
#include "seqattn.h"

namespace seqattn {

// One error word per device (see sm103_ptx.cuh, "device error word").
__device__ unsigned int g_seqattn_error_word = 0u;

namespace {

thread_local std::string t_last_error;

seqattn_status fail(seqattn_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
seqattn_status fail(seqattn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return s;
}

seqattn_status ok() {
  t_last_error.clear();
  return SEQATTN_OK;
}

seqattn_status cuda_fail(cudaError_t e, const char* where) {
  return fail(SEQATTN_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;
std::mutex g_mu;
unsigned int* g_err_ptr[kMaxDevices] = {};

// Limit of every bounded device wait of the kernels launched from now on
// (seqattn_set_wait_limit); the default is about one second.
constexpr long long kDefaultWaitCycles = 2000000000LL;
std::atomic<long long> g_wait_cycles{kDefaultWaitCycles};

// Device address of this device's error word (looked up once per device).
cudaError_t error_word(unsigned int** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_err_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_seqattn_error_word);
    if (e != cudaSuccess) return e;
    g_err_ptr[dev] = static_cast<unsigned int*>(p);
  }
  *out = g_err_ptr[dev];
  return cudaSuccess;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// 3-D bf16 tensor map over a [rows, heads, d] row-major tensor: box of
// {64 elements of d, 1 head, box_rows rows}, 128-byte swizzle (one 128-byte
// row of the box per smem row, the layout the MMA descriptors expect).
bool make_map(CUtensorMap* m, const void* base, int d, int heads, int64_t rows, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  memset(m, 0, sizeof(*m));
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                           static_cast<cuuint64_t>(heads) * static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D tensor map over a row-major [B, T, cols] tensor of bf16 (128-byte
// swizzle, box {64 columns, box_rows rows, 1 batch entry}) or float32 (no
// swizzle, box {box_cols, box_rows, 1}).  Rows past T and columns past
// `cols` read as zero and are never written.
bool make_map_btc(CUtensorMap* m, const void* base, int64_t B, int64_t T, int64_t cols, bool fp32,
                  int box_cols, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  memset(m, 0, sizeof(*m));
  const cuuint64_t es_bytes = fp32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * es_bytes,
                           static_cast<cuuint64_t>(T) * static_cast<cuuint64_t>(cols) * es_bytes};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  fp32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 4-D float32 tensor map over the [B, T, heads, d] accumulator, cut at row
// `rows` of every batch entry (the chunk's end: rows past it are never
// written): box {32 of d, 1 head, 128 rows, 1 batch entry}, 128-byte swizzle.
bool make_map_accum(CUtensorMap* m, const void* base, int d, int heads, int64_t T, int64_t rows, int B) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  memset(m, 0, sizeof(*m));
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 4, static_cast<cuuint64_t>(heads) * d * 4,
                           static_cast<cuuint64_t>(T) * heads * d * 4};
  cuuint32_t box[4] = {32, 1, 128, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

seqattn_status check_problem(const seqattn_problem* pb) {
  if (pb == nullptr) return fail(SEQATTN_ERR_INVALID_ARG, "problem is NULL");
  if (pb->batch < 1 || pb->num_q_heads < 1 || pb->num_kv_heads < 1 || pb->seq_capacity < 1)
    return fail(SEQATTN_ERR_INVALID_ARG, "batch, heads and seq_capacity must be >= 1");
  if (pb->num_q_heads % pb->num_kv_heads != 0)
    return fail(SEQATTN_ERR_INVALID_ARG, "num_q_heads (%d) is not a multiple of num_kv_heads (%d)",
                pb->num_q_heads, pb->num_kv_heads);
  if (pb->head_dim != 64 && pb->head_dim != 128)
    return fail(SEQATTN_ERR_INVALID_ARG, "head_dim %d is not 64 or 128", pb->head_dim);
  if (pb->dtype != SEQATTN_BF16 && pb->dtype != SEQATTN_FP32)
    return fail(SEQATTN_ERR_INVALID_ARG, "unknown dtype %d", pb->dtype);
  if (static_cast<int64_t>(pb->batch) * pb->seq_capacity > INT32_MAX)
    return fail(SEQATTN_ERR_INVALID_ARG, "batch * seq_capacity exceeds 2^31 - 1 rows");
  return SEQATTN_OK;
}

seqattn_status check_chunk(const seqattn_problem* pb, int64_t q_start, int64_t q_len,
                           int64_t prefix_len, float scale, ChunkGeom* g) {
  seqattn_status s = check_problem(pb);
  if (s != SEQATTN_OK) return s;
  if (q_len < 0) return fail(SEQATTN_ERR_INVALID_ARG, "q_len %lld < 0", (long long)q_len);
  if (q_start < 0 || prefix_len < 0 || prefix_len > q_start)
    return fail(SEQATTN_ERR_INVALID_ARG, "need 0 <= prefix_len <= q_start (got %lld, %lld)",
                (long long)prefix_len, (long long)q_start);
  if (q_start > pb->seq_capacity || q_len > pb->seq_capacity - q_start)     // (their sum may pass int64)
    return fail(SEQATTN_ERR_INVALID_ARG, "q_start + q_len = %lld + %lld exceeds seq_capacity %lld", (long long)q_start,
                (long long)q_len, (long long)pb->seq_capacity);
  if (!(scale > 0.f) || !isfinite(scale))
    return fail(SEQATTN_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  if (static_cast<int64_t>(pb->batch) * q_len > INT32_MAX)
    return fail(SEQATTN_ERR_INVALID_ARG, "batch * q_len exceeds 2^31 - 1 rows");
  g->B = pb->batch;
  g->Hq = pb->num_q_heads;
  g->Hkv = pb->num_kv_heads;
  g->G = pb->num_q_heads / pb->num_kv_heads;
  g->d = pb->head_dim;
  g->T = pb->seq_capacity;
  g->q_start = q_start;
  g->q_len = q_len;
  g->kv_begin = q_start - prefix_len;
  g->scale = scale;
  g->wait_cycles = g_wait_cycles.load(std::memory_order_relaxed);
  return SEQATTN_OK;
}

seqattn_status check_ptrs(std::initializer_list<std::pair<const void*, const char*>> ps) {
  for (auto& p : ps) {
    if (p.first == nullptr) return fail(SEQATTN_ERR_INVALID_ARG, "%s is NULL", p.second);
    if (!aligned16(p.first))
      return fail(SEQATTN_ERR_INVALID_ARG, "%s is not 16-byte aligned", p.second);
  }
  return SEQATTN_OK;
}

size_t workspace_bytes(const seqattn_problem* pb, int64_t q_len) {
  // float32: Delta [B, Hq, q_len].  bf16: -L log2(e) and Delta per 64-row
  // query tile, [B, Hq, ceil(q_len / 64), 2, 64].  Rounded up to 256 bytes.
  const size_t rows = pb->dtype == SEQATTN_BF16 ? static_cast<size_t>((q_len + 63) / 64) * 128
                                                : static_cast<size_t>(q_len);
  const size_t bytes = static_cast<size_t>(pb->batch) * pb->num_q_heads * rows * sizeof(float);
  return (bytes + 255) & ~static_cast<size_t>(255);
}

}  // namespace
}  // namespace seqattn

using namespace seqattn;

extern "C" {

seqattn_status seqattn_chunk_fwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len,
                                 int64_t prefix_len, float softmax_scale, const void* q,
                                 const void* k, const void* v, void* o, float* lse,
                                 seqattn_stream_t stream) {
  ChunkGeom g;
  seqattn_status s = check_chunk(pb, q_start, q_len, prefix_len, softmax_scale, &g);
  if (s != SEQATTN_OK) return s;
  if (q_len == 0) return ok();
  s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {o, "o"}, {lse, "lse"}});
  if (s != SEQATTN_OK) return s;
  unsigned int* err = nullptr;
  cudaError_t e = error_word(&err);
  if (e != cudaSuccess) return cuda_fail(e, "error word");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (pb->dtype == SEQATTN_FP32) {
    e = launch_fwd_f32(g, static_cast<const float*>(q), static_cast<const float*>(k),
                       static_cast<const float*>(v), static_cast<float*>(o), lse, err, st);
    return e == cudaSuccess ? ok() : cuda_fail(e, "fwd_f32 launch");
  }
  Bf16FwdMaps maps;
  if (!make_map(&maps.q, q, g.d, g.Hq, static_cast<int64_t>(g.B) * q_len, 128) ||
      !make_map(&maps.k, k, g.d, g.Hkv, static_cast<int64_t>(g.B) * g.T, 128) ||
      !make_map(&maps.v, v, g.d, g.Hkv, static_cast<int64_t>(g.B) * g.T, 128))
    return fail(SEQATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed for the forward operands");
  e = launch_fwd_bf16(g, maps, o, lse, err, st);
  return e == cudaSuccess ? ok() : cuda_fail(e, "fwd_bf16 launch");
}

seqattn_status seqattn_chunk_bwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len,
                                 int64_t prefix_len, float softmax_scale, const void* q,
                                 const void* k, const void* v, const void* o, const float* lse,
                                 const void* d_o, float* dq, float* dk_accum, float* dv_accum,
                                 void* workspace, size_t workspace_size, seqattn_stream_t stream) {
  ChunkGeom g;
  seqattn_status s = check_chunk(pb, q_start, q_len, prefix_len, softmax_scale, &g);
  if (s != SEQATTN_OK) return s;
  if (q_len == 0) return ok();
  s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {o, "o"}, {lse, "lse"}, {d_o, "d_o"}, {dq, "dq"},
                  {dk_accum, "dk_accum"}, {dv_accum, "dv_accum"}, {workspace, "workspace"}});
  if (s != SEQATTN_OK) return s;
  if (workspace_size < workspace_bytes(pb, q_len))
    return fail(SEQATTN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed",
                workspace_size, workspace_bytes(pb, q_len));
  unsigned int* err = nullptr;
  cudaError_t e = error_word(&err);
  if (e != cudaSuccess) return cuda_fail(e, "error word");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  float* delta = static_cast<float*>(workspace);
  if (pb->dtype == SEQATTN_FP32) {
    e = launch_bwd_prep_f32(g, static_cast<const float*>(o), static_cast<const float*>(d_o), delta,
                            st);
    if (e != cudaSuccess) return cuda_fail(e, "bwd_prep launch");
    e = launch_bwd_f32(g, static_cast<const float*>(q), static_cast<const float*>(k),
                       static_cast<const float*>(v), lse, static_cast<const float*>(d_o), delta,
                       dq, dk_accum, dv_accum, err, st);
    return e == cudaSuccess ? ok() : cuda_fail(e, "bwd_f32 launch");
  }
  Bf16BwdMaps maps;
  if (!make_map(&maps.q, q, g.d, g.Hq, static_cast<int64_t>(g.B) * q_len, 64) ||
      !make_map(&maps.d_o, d_o, g.d, g.Hq, static_cast<int64_t>(g.B) * q_len, 64) ||
      !make_map(&maps.k, k, g.d, g.Hkv, static_cast<int64_t>(g.B) * g.T, 128) ||
      !make_map(&maps.v, v, g.d, g.Hkv, static_cast<int64_t>(g.B) * g.T, 128) ||
      !make_map_accum(&maps.dk, dk_accum, g.d, g.Hkv, g.T, q_start + q_len, g.B) ||
      !make_map_accum(&maps.dv, dv_accum, g.d, g.Hkv, g.T, q_start + q_len, g.B))
    return fail(SEQATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed for the backward operands");
  e = launch_bwd_stats_bf16(g, o, d_o, lse, delta, dq, st);
  if (e != cudaSuccess) return cuda_fail(e, "bwd_stats launch");
  e = launch_bwd_bf16(g, maps, delta, dq, dk_accum, dv_accum, err, st);
  return e == cudaSuccess ? ok() : cuda_fail(e, "bwd_bf16 launch");
}

seqattn_status seqattn_reset_accum(const seqattn_problem* pb, float* dk_accum, float* dv_accum,
                                   seqattn_stream_t stream) {
  seqattn_status s = check_problem(pb);
  if (s != SEQATTN_OK) return s;
  s = check_ptrs({{dk_accum, "dk_accum"}, {dv_accum, "dv_accum"}});
  if (s != SEQATTN_OK) return s;
  const int64_t n = static_cast<int64_t>(pb->batch) * pb->seq_capacity * pb->num_kv_heads *
                    pb->head_dim;
  cudaError_t e = launch_zero_f32(dk_accum, dv_accum, n, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "reset launch");
}

seqattn_status seqattn_scale_accum_rows(const seqattn_problem* pb, int64_t row_begin,
                                        int64_t row_end, float scale, float* dk_accum,
                                        float* dv_accum, seqattn_stream_t stream) {
  seqattn_status s = check_problem(pb);
  if (s != SEQATTN_OK) return s;
  if (row_begin < 0 || row_end < row_begin || row_end > pb->seq_capacity)
    return fail(SEQATTN_ERR_INVALID_ARG, "need 0 <= row_begin <= row_end <= seq_capacity (got %lld, %lld)",
                (long long)row_begin, (long long)row_end);
  if (!isfinite(scale)) return fail(SEQATTN_ERR_INVALID_ARG, "scale must be finite");
  s = check_ptrs({{dk_accum, "dk_accum"}, {dv_accum, "dv_accum"}});
  if (s != SEQATTN_OK) return s;
  cudaError_t e = launch_scale_rows_f32(dk_accum, dv_accum, pb->batch, pb->seq_capacity, row_begin, row_end,
                                        static_cast<int64_t>(pb->num_kv_heads) * pb->head_dim, scale,
                                        reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "scale launch");
}

seqattn_status seqattn_proj_wgrad(int32_t batch, int64_t seq_len, int64_t row_begin,
                                  int64_t row_end, int32_t d_model, int32_t n, const void* h,
                                  const float* g, float* dw, seqattn_stream_t stream) {
  if (batch < 1 || seq_len < 1) return fail(SEQATTN_ERR_INVALID_ARG, "batch and seq_len must be >= 1");
  if (row_begin < 0 || row_end < row_begin || row_end > seq_len)
    return fail(SEQATTN_ERR_INVALID_ARG, "need 0 <= row_begin <= row_end <= seq_len (got %lld, %lld)",
                (long long)row_begin, (long long)row_end);
  if (d_model < 8 || d_model % 8 || n < 8 || n % 8)
    return fail(SEQATTN_ERR_INVALID_ARG, "d_model (%d) and n (%d) must be positive multiples of 8", d_model, n);
  if (static_cast<int64_t>(batch) * seq_len > INT32_MAX || seq_len * static_cast<int64_t>(n) > INT32_MAX)
    return fail(SEQATTN_ERR_INVALID_ARG, "batch * seq_len or seq_len * n exceeds 2^31 - 1");
  seqattn_status s = check_ptrs({{h, "h"}, {g, "g"}, {dw, "dw"}});
  if (s != SEQATTN_OK) return s;
  if (row_end == row_begin) return ok();
  unsigned int* err = nullptr;
  cudaError_t e = error_word(&err);
  if (e != cudaSuccess) return cuda_fail(e, "error word");
  WgradMaps maps;
  if (!make_map_btc(&maps.h, h, batch, seq_len, d_model, false, 64, kWgradStageRows) ||
      !make_map_btc(&maps.g, g, batch, seq_len, n, true, 128, kWgradStageRows) ||
      !make_map_btc(&maps.dw, dw, 1, d_model, n, true, 128, 32))
    return fail(SEQATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed for h, g or dw");
  e = launch_wgrad_bf16(maps, batch, row_begin, row_end, d_model, n, err,
                        g_wait_cycles.load(std::memory_order_relaxed), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "wgrad launch");
}

size_t seqattn_bwd_workspace_size(const seqattn_problem* pb, int64_t q_len) {
  if (check_problem(pb) != SEQATTN_OK || q_len < 0) return 0;
  return workspace_bytes(pb, q_len);
}

seqattn_status seqattn_sync_status(seqattn_stream_t stream) {
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  unsigned int* err = nullptr;
  if ((e = error_word(&err)) != cudaSuccess) return cuda_fail(e, "error word");
  unsigned int w = 0;
  if ((e = cudaMemcpy(&w, err, sizeof(w), cudaMemcpyDeviceToHost)) != cudaSuccess)
    return cuda_fail(e, "read error word");
  if (w != 0) {
    const unsigned int zero = 0;
    if ((e = cudaMemcpy(err, &zero, sizeof(zero), cudaMemcpyHostToDevice)) != cudaSuccess)
      return cuda_fail(e, "clear error word");
    return fail(SEQATTN_ERR_TIMEOUT, "a kernel gave up a bounded wait (error word 0x%x)", w);
  }
  return ok();
}

void seqattn_set_wait_limit(int64_t cycles) {
  g_wait_cycles.store(cycles > 0 ? cycles : kDefaultWaitCycles, std::memory_order_relaxed);
}

const char* seqattn_status_string(seqattn_status s) {
  switch (s) {
    case SEQATTN_OK: return "ok";
    case SEQATTN_ERR_INVALID_ARG: return "invalid argument";
    case SEQATTN_ERR_UNSUPPORTED: return "unsupported";
    case SEQATTN_ERR_CUDA: return "CUDA error";
    case SEQATTN_ERR_TIMEOUT: return "device wait timed out";
  }
  return "unknown status";
}

const char* seqattn_last_error(void) { return t_last_error.c_str(); }

}  // extern "C"

// ---------------------------------------------------------------------------
// Backward for callers that cannot allocate device memory.
//
// Some callers have no way to provide the backward's scratch buffer: their
// device memory is owned by another allocator (a framework's caching
// allocator or a fixed arena handed out at start-up) and the plugin interface
// they call through passes only the tensors themselves.  For them the Delta
// scratch lives in a fixed array in this file, so the call needs nothing
// beyond its inputs and outputs.
// ---------------------------------------------------------------------------
namespace seqattn {
namespace {

// Row-statistics scratch (what seqattn_bwd_workspace_size asks for, at most
// 4 MiB) on every GPU that loads the library, held until the process exits.
static __device__ __align__(256) float g_noalloc_delta[SEQATTN_NOALLOC_MAX_DELTA];

float* g_noalloc_ptr[kMaxDevices] = {};

// Device address of this device's scratch array.  Host code cannot use the
// array's name as a device pointer, so the address is looked up once per
// device, with that device current, on the first call there.
cudaError_t noalloc_scratch(float** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_delta);
    if (e != cudaSuccess) return e;
    g_noalloc_ptr[dev] = static_cast<float*>(p);
  }
  *out = g_noalloc_ptr[dev];
  return cudaSuccess;
}

}  // namespace
}  // namespace seqattn

extern "C" seqattn_status seqattn_chunk_bwd_noalloc(
    const seqattn_problem* pb, int64_t q_start, int64_t q_len, int64_t prefix_len,
    float softmax_scale, const void* q, const void* k, const void* v, const void* o,
    const float* lse, const void* d_o, float* dq, float* dk_accum, float* dv_accum,
    seqattn_stream_t stream) {
  ChunkGeom g;
  seqattn_status s = check_chunk(pb, q_start, q_len, prefix_len, softmax_scale, &g);
  if (s != SEQATTN_OK) return s;
  if (q_len == 0) return ok();
  s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {o, "o"}, {lse, "lse"}, {d_o, "d_o"}, {dq, "dq"},
                  {dk_accum, "dk_accum"}, {dv_accum, "dv_accum"}});
  if (s != SEQATTN_OK) return s;
  const size_t need = workspace_bytes(pb, q_len);
  if (need > sizeof(float) * static_cast<size_t>(SEQATTN_NOALLOC_MAX_DELTA))
    return fail(SEQATTN_ERR_INVALID_ARG,
                "this chunk needs %zu bytes of row statistics, more than the fixed scratch of %d "
                "floats of seqattn_chunk_bwd_noalloc; use seqattn_chunk_bwd with a workspace",
                need, SEQATTN_NOALLOC_MAX_DELTA);
  float* delta = nullptr;
  cudaError_t e = noalloc_scratch(&delta);
  if (e != cudaSuccess) return cuda_fail(e, "scratch address");
  unsigned int* err = nullptr;
  if ((e = error_word(&err)) != cudaSuccess) return cuda_fail(e, "error word");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (pb->dtype == SEQATTN_FP32) {
    e = launch_bwd_prep_f32(g, static_cast<const float*>(o), static_cast<const float*>(d_o), delta,
                            st);
    if (e != cudaSuccess) return cuda_fail(e, "bwd_prep launch");
    e = launch_bwd_f32(g, static_cast<const float*>(q), static_cast<const float*>(k),
                       static_cast<const float*>(v), lse, static_cast<const float*>(d_o), delta,
                       dq, dk_accum, dv_accum, err, st);
    return e == cudaSuccess ? ok() : cuda_fail(e, "bwd_f32 launch");
  }
  Bf16BwdMaps maps;
  if (!make_map(&maps.q, q, g.d, g.Hq, static_cast<int64_t>(g.B) * q_len, 64) ||
      !make_map(&maps.d_o, d_o, g.d, g.Hq, static_cast<int64_t>(g.B) * q_len, 64) ||
      !make_map(&maps.k, k, g.d, g.Hkv, static_cast<int64_t>(g.B) * g.T, 128) ||
      !make_map(&maps.v, v, g.d, g.Hkv, static_cast<int64_t>(g.B) * g.T, 128) ||
      !make_map_accum(&maps.dk, dk_accum, g.d, g.Hkv, g.T, q_start + q_len, g.B) ||
      !make_map_accum(&maps.dv, dv_accum, g.d, g.Hkv, g.T, q_start + q_len, g.B))
    return fail(SEQATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed for the backward operands");
  e = launch_bwd_stats_bf16(g, o, d_o, lse, delta, dq, st);
  if (e != cudaSuccess) return cuda_fail(e, "bwd_stats launch");
  e = launch_bwd_bf16(g, maps, delta, dq, dk_accum, dv_accum, err, st);
  return e == cudaSuccess ? ok() : cuda_fail(e, "bwd_bf16 launch");
}

// ---------------------------------------------------------------------------
// The rest of the layer: linear products, head norm + rotary positions, AdamW.
// ---------------------------------------------------------------------------
namespace seqattn {
namespace {

// What L2 fetches for a 128-byte row of a box.  A row that starts off a
// 128-byte line touches two, and fetching 256 bytes for each costs time
// (512 x 4104 x 10248: 51 us, 47 with 128 bytes); on whole lines 256 bytes read
// memory a little faster (2048 x 4096 x 4096 from a cold L2: 50.8 us, 51.3 with 128).
CUtensorMapL2promotion promotion(int64_t ld) {
  return ld % 64 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
}

// 2-D bf16 tensor map over a row-major [rows, cols] matrix with a row stride
// of `ld` elements: box {64 columns, box_rows rows}, 128-byte swizzle; reads
// past the matrix give zeros.
bool make_map_2d(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  memset(m, 0, sizeof(*m));
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion(ld),
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The same matrix with its 64-column blocks as a third dimension (cols a
// multiple of 64): box {64 columns, 64 rows, 2 blocks}.
bool make_map_blocks(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  memset(m, 0, sizeof(*m));
  cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, 128};
  cuuint32_t box[3] = {64, kLinearStageK, 2};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion(ld),
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 2-D map over a dense float32 [rows, cols] matrix: box {32, 32}, 128-byte swizzle.
bool make_map_f32(CUtensorMap* m, const void* base, int64_t rows, int64_t cols) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  memset(m, 0, sizeof(*m));
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 4};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

seqattn_status check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld % 8 != 0 || ld > (int64_t{1} << 36))
    return fail(SEQATTN_ERR_INVALID_ARG, "row stride of %s (%lld) must be a multiple of 8 and at least %lld", name,
                (long long)ld, (long long)cols);
  return SEQATTN_OK;
}

seqattn_status check_linear(int64_t rows, int32_t k, int32_t n, int32_t act) {
  if (rows < 0 || rows >= INT32_MAX - 511)
    return fail(SEQATTN_ERR_INVALID_ARG, "rows (%lld) must lie in [0, 2^31 - 512)", (long long)rows);
  if (k < 8 || k % 8 || n < 8 || n % 8 || k > INT32_MAX - 511 || n > INT32_MAX - 511)
    return fail(SEQATTN_ERR_INVALID_ARG, "k (%d) and n (%d) must be positive multiples of 8", k, n);
  if (act < SEQATTN_ACT_NONE || act > SEQATTN_ACT_GELU_TANH)
    return fail(SEQATTN_ERR_INVALID_ARG, "unknown activation %d", act);
  return SEQATTN_OK;
}

// Refuses outputs that start where another operand does: in-place calls that
// the kernels, whose tiles are written while others are still read, cannot make.
seqattn_status check_apart(std::initializer_list<std::pair<const void*, const char*>> outs,
                           std::initializer_list<std::pair<const void*, const char*>> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (o->first == nullptr) continue;
    for (auto other = o + 1; other != outs.end(); ++other)
      if (o->first == other->first)
        return fail(SEQATTN_ERR_INVALID_ARG, "%s and %s are the same memory", o->second, other->second);
    for (auto& in : ins)
      if (o->first == in.first)
        return fail(SEQATTN_ERR_INVALID_ARG, "%s is the memory of %s", o->second, in.second);
  }
  return SEQATTN_OK;
}

// The residual may be the output itself, element for element.
seqattn_status check_residual(const void* residual, int64_t ldr, const void* out, int64_t ldo) {
  if (residual != nullptr && residual == out && ldr != ldo)
    return fail(SEQATTN_ERR_INVALID_ARG, "the residual is the output with another row stride (%lld, %lld)", (long long)ldr,
                (long long)ldo);
  return SEQATTN_OK;
}

// Common end of the three linear calls: error word, wait limit, maps, launch.
// Operand a carries the result's row index, b its column index.  An operand
// whose contiguous dimension is that index (MN-major) is `mn` columns of
// contraction rows, of the other kind (K-major) `mn` rows.
seqattn_status run_linear(int mode, LinearParams& p, const void* a, int64_t lda, const void* b, int64_t ldb,
                          seqattn_stream_t stream) {
  unsigned int* err = nullptr;
  cudaError_t e = error_word(&err);
  if (e != cudaSuccess) return cuda_fail(e, "error word");
  p.err = err;
  p.wait_cycles = g_wait_cycles.load(std::memory_order_relaxed);
  if (mode == kLinearFwd && p.m <= kLinearGemvRows) {
    e = launch_linear_gemv(p, a, lda, b, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, "linear launch");
  }
  if ((e = plan_linear_bf16(mode, p)) != cudaSuccess) return cuda_fail(e, "linear plan");
  LinearMaps maps;
  memset(&maps.out, 0, sizeof(maps.out));
  // whole blocks only, and tiles (halves of a pair's) that start on one
  auto mn_map = [&](CUtensorMap* m, const void* base, int64_t mn, int64_t ld, int* blocked) {
    *blocked = mn % 64 == 0 && p.tile_n % 128 == 0;
    return *blocked ? make_map_blocks(m, base, p.k, mn, ld) : make_map_2d(m, base, p.k, mn, ld, kLinearStageK);
  };
  const bool made = (mode == kLinearWgrad ? mn_map(&maps.a, a, p.m, lda, &p.a_blocked)
                                          : make_map_2d(&maps.a, a, p.m, p.k, lda, linear_a_rows(p.m))) &&
                    (mode != kLinearDgrad ? mn_map(&maps.b, b, p.n, ldb, &p.b_blocked)
                                          : make_map_2d(&maps.b, b, p.n, p.k, ldb, 128)) &&
                    (mode != kLinearWgrad || make_map_f32(&maps.out, p.out, p.m, p.n));
  if (!made) return fail(SEQATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed for the operands of the product");
  e = launch_linear_bf16(mode, maps, p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "linear launch");
}

}  // namespace
}  // namespace seqattn

extern "C" {

seqattn_status seqattn_linear_fwd(int64_t rows, int32_t k, int32_t n, const void* x, int64_t ldx, const void* w,
                                  const void* bias, int32_t act, const void* residual, int64_t ldr, void* z,
                                  int64_t ldz, void* y, int64_t ldy, seqattn_stream_t stream) {
  seqattn_status s = check_linear(rows, k, n, act);
  if (s != SEQATTN_OK) return s;
  if ((s = check_ld(ldx, k, "x")) != SEQATTN_OK || (s = check_ld(ldy, n, "y")) != SEQATTN_OK) return s;
  if (residual != nullptr && (s = check_ld(ldr, n, "residual")) != SEQATTN_OK) return s;
  if (z != nullptr && (s = check_ld(ldz, n, "z")) != SEQATTN_OK) return s;
  if (rows == 0) return ok();
  s = check_ptrs({{x, "x"}, {w, "w"}, {y, "y"}});
  if (s != SEQATTN_OK) return s;
  if (!aligned16(bias) || !aligned16(residual) || !aligned16(z))
    return fail(SEQATTN_ERR_INVALID_ARG, "bias, residual or z is not 16-byte aligned");
  if ((s = check_apart({{y, "y"}, {z, "z"}}, {{x, "x"}, {w, "w"}, {bias, "bias"}})) != SEQATTN_OK ||
      (s = check_apart({{z, "z"}}, {{residual, "residual"}})) != SEQATTN_OK ||
      (s = check_residual(residual, ldr, y, ldy)) != SEQATTN_OK)
    return s;
  LinearParams p = {};
  p.m = static_cast<int>(rows);
  p.n = n;
  p.k = k;
  p.act = act;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.z = static_cast<__nv_bfloat16*>(z);
  p.out = y;
  p.ldr = ldr;
  p.ldz = ldz;
  p.ldo = ldy;
  return run_linear(kLinearFwd, p, x, ldx, w, n, stream);
}

seqattn_status seqattn_linear_dgrad(int64_t rows, int32_t k, int32_t n, const void* g, int64_t ldg, const void* w,
                                    int32_t act, const void* z, int64_t ldz, const void* residual, int64_t ldr,
                                    void* dx, int64_t lddx, seqattn_stream_t stream) {
  seqattn_status s = check_linear(rows, k, n, act);
  if (s != SEQATTN_OK) return s;
  if ((s = check_ld(ldg, n, "g")) != SEQATTN_OK || (s = check_ld(lddx, k, "dx")) != SEQATTN_OK) return s;
  if (residual != nullptr && (s = check_ld(ldr, k, "residual")) != SEQATTN_OK) return s;
  if (act != SEQATTN_ACT_NONE) {
    if (z == nullptr && rows > 0) return fail(SEQATTN_ERR_INVALID_ARG, "z is NULL but act is not NONE");
    if ((s = check_ld(ldz, k, "z")) != SEQATTN_OK) return s;
  }
  if (rows == 0) return ok();
  s = check_ptrs({{g, "g"}, {w, "w"}, {dx, "dx"}});
  if (s != SEQATTN_OK) return s;
  if (!aligned16(residual) || !aligned16(z))
    return fail(SEQATTN_ERR_INVALID_ARG, "residual or z is not 16-byte aligned");
  if ((s = check_apart({{dx, "dx"}}, {{g, "g"}, {w, "w"}, {act != SEQATTN_ACT_NONE ? z : nullptr, "z"}})) != SEQATTN_OK ||
      (s = check_residual(residual, ldr, dx, lddx)) != SEQATTN_OK)
    return s;
  LinearParams p = {};
  p.m = static_cast<int>(rows);
  p.n = k;
  p.k = n;
  p.act = act;
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.z = static_cast<__nv_bfloat16*>(const_cast<void*>(z));   // read only by dgrad
  p.out = dx;
  p.ldr = ldr;
  p.ldz = ldz;
  p.ldo = lddx;
  return run_linear(kLinearDgrad, p, g, ldg, w, n, stream);
}

seqattn_status seqattn_linear_wgrad(int64_t rows, int32_t k, int32_t n, const void* x, int64_t ldx, const void* g,
                                    int64_t ldg, float* dw, float* dbias, seqattn_stream_t stream) {
  seqattn_status s = check_linear(rows, k, n, SEQATTN_ACT_NONE);
  if (s != SEQATTN_OK) return s;
  if ((s = check_ld(ldx, k, "x")) != SEQATTN_OK || (s = check_ld(ldg, n, "g")) != SEQATTN_OK) return s;
  if (rows == 0) return ok();
  s = check_ptrs({{x, "x"}, {g, "g"}, {dw, "dw"}});
  if (s != SEQATTN_OK) return s;
  if (!aligned16(dbias)) return fail(SEQATTN_ERR_INVALID_ARG, "dbias is not 16-byte aligned");
  if ((s = check_apart({{dw, "dw"}, {dbias, "dbias"}}, {{x, "x"}, {g, "g"}})) != SEQATTN_OK) return s;
  LinearParams p = {};
  p.m = k;
  p.n = n;
  p.k = static_cast<int>(rows);
  p.out = dw;
  p.ldo = n;
  s = run_linear(kLinearWgrad, p, x, ldx, g, ldg, stream);
  if (s != SEQATTN_OK || dbias == nullptr) return s;
  const cudaError_t e =
      launch_colsum_bf16(g, ldg, static_cast<int>(rows), n, dbias, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "column sum launch");
}

}  // extern "C"

namespace seqattn {
namespace {

// The checks that the forward and the backward of the head norm share, and
// the part of the launch parameters that they fill.
seqattn_status check_norm_rope(const seqattn_problem* pb, int64_t q_start, int64_t q_len, const void* gamma_q,
                               const void* gamma_k, float eps, const seqattn_rope_plan* plan,
                               const int64_t* positions, NormRopeParams* p) {
  seqattn_status s = check_problem(pb);
  if (s != SEQATTN_OK) return s;
  if (q_start < 0 || q_len < 0 || q_start > pb->seq_capacity || q_len > pb->seq_capacity - q_start)
    return fail(SEQATTN_ERR_INVALID_ARG, "need 0 <= q_start and 0 <= q_len and q_start + q_len <= seq_capacity (got %lld, %lld)",
                (long long)q_start, (long long)q_len);
  if (static_cast<int64_t>(pb->num_q_heads) * pb->head_dim > INT32_MAX)
    return fail(SEQATTN_ERR_INVALID_ARG, "num_q_heads * head_dim exceeds 2^31 - 1");
  if ((gamma_q == nullptr) != (gamma_k == nullptr))
    return fail(SEQATTN_ERR_INVALID_ARG, "gamma_q and gamma_k must both be given or both be NULL");
  if (gamma_q != nullptr && !(eps >= 0.f && isfinite(eps)))
    return fail(SEQATTN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!aligned16(gamma_q) || !aligned16(gamma_k))
    return fail(SEQATTN_ERR_INVALID_ARG, "gamma is not 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(positions) & 7u) != 0)
    return fail(SEQATTN_ERR_INVALID_ARG, "positions is not 8-byte aligned");
  p->B = pb->batch;
  p->q_len = static_cast<int>(q_len);
  p->Hq = pb->num_q_heads;
  p->Hkv = pb->num_kv_heads;
  p->T = pb->seq_capacity;
  p->q_start = q_start;
  p->gamma_q = gamma_q;
  p->gamma_k = gamma_k;
  p->eps = eps;
  p->positions = positions;
  p->rot_dim = 0;
  if (plan != nullptr) {
    if (plan->rot_dim < 16 || plan->rot_dim % 16 || plan->rot_dim > pb->head_dim)
      return fail(SEQATTN_ERR_INVALID_ARG, "rot_dim %d is not a multiple of 16 in [16, head_dim]", plan->rot_dim);
    if (plan->axes < 1 || plan->axes > 64 || (plan->interleaved != 0 && plan->interleaved != 1) ||
        plan->reserved != 0)
      return fail(SEQATTN_ERR_INVALID_ARG, "rope plan: axes must lie in [1, 64], interleaved be 0 or 1, reserved 0");
    for (int i = 0; i < plan->rot_dim / 2; ++i)
      if (plan->axis[i] >= plan->axes)
        return fail(SEQATTN_ERR_INVALID_ARG, "rope plan: axis[%d] = %d is not below axes = %d", i, plan->axis[i],
                    plan->axes);
    p->rot_dim = plan->rot_dim;
    p->axes = plan->axes;
    p->interleaved = plan->interleaved;
    memcpy(p->turns, plan->turns, sizeof(p->turns));
    memcpy(p->axis, plan->axis, sizeof(p->axis));
  }
  return SEQATTN_OK;
}

size_t norm_rope_workspace(int head_dim) {
  return static_cast<size_t>(norm_rope_bwd_blocks()) * 2 * head_dim * sizeof(float);
}

}  // namespace
}  // namespace seqattn

extern "C" {

seqattn_status seqattn_qk_norm_rope_fwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len, const void* q_in,
                                        int64_t ld_q, const void* k_in, int64_t ld_k, const void* v_in, int64_t ld_v,
                                        const void* gamma_q, const void* gamma_k, float eps,
                                        const seqattn_rope_plan* plan, const int64_t* positions, void* q,
                                        void* k_cache, void* v_cache, seqattn_stream_t stream) {
  NormRopeParams p = {};
  seqattn_status s = check_norm_rope(pb, q_start, q_len, gamma_q, gamma_k, eps, plan, positions, &p);
  if (s != SEQATTN_OK) return s;
  const int64_t nq = static_cast<int64_t>(pb->num_q_heads) * pb->head_dim;
  const int64_t nk = static_cast<int64_t>(pb->num_kv_heads) * pb->head_dim;
  if ((v_in == nullptr) != (v_cache == nullptr))
    return fail(SEQATTN_ERR_INVALID_ARG, "v_in and v_cache must both be given or both be NULL");
  if ((s = check_ld(ld_q, nq, "q_in")) != SEQATTN_OK || (s = check_ld(ld_k, nk, "k_in")) != SEQATTN_OK) return s;
  if (v_in != nullptr && (s = check_ld(ld_v, nk, "v_in")) != SEQATTN_OK) return s;
  if (q_len == 0) return ok();
  s = check_ptrs({{q_in, "q_in"}, {k_in, "k_in"}, {q, "q"}, {k_cache, "k_cache"}});
  if (s != SEQATTN_OK) return s;
  if (!aligned16(v_in) || !aligned16(v_cache))
    return fail(SEQATTN_ERR_INVALID_ARG, "v_in or v_cache is not 16-byte aligned");
  s = check_apart({{q, "q"}, {k_cache, "k_cache"}, {v_cache, "v_cache"}},
                  {{q_in, "q_in"}, {k_in, "k_in"}, {v_in, "v_in"}, {gamma_q, "gamma_q"}, {gamma_k, "gamma_k"}});
  if (s != SEQATTN_OK) return s;
  p.q_in = q_in;
  p.k_in = k_in;
  p.v_in = v_in;
  p.q_stride = ld_q;
  p.k_stride = ld_k;
  p.v_stride = ld_v;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  const cudaError_t e = launch_norm_rope_fwd(p, pb->head_dim, pb->dtype == SEQATTN_BF16,
                                             reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "norm_rope_fwd launch");
}

size_t seqattn_qk_norm_rope_bwd_workspace_size(const seqattn_problem* pb) {
  return check_problem(pb) == SEQATTN_OK ? norm_rope_workspace(pb->head_dim) : 0;
}

seqattn_status seqattn_qk_norm_rope_bwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len, const void* q_in,
                                        int64_t ld_q, const void* k_in, int64_t ld_k, const void* gamma_q,
                                        const void* gamma_k, float eps, const seqattn_rope_plan* plan,
                                        const int64_t* positions, const float* dq, const float* dk_accum,
                                        const float* dv_accum, void* dq_in, int64_t ld_dq, void* dk_in,
                                        int64_t ld_dk, void* dv_in, int64_t ld_dv, float* dgamma_q, float* dgamma_k,
                                        void* workspace, size_t workspace_size, seqattn_stream_t stream) {
  NormRopeParams p = {};
  seqattn_status s = check_norm_rope(pb, q_start, q_len, gamma_q, gamma_k, eps, plan, positions, &p);
  if (s != SEQATTN_OK) return s;
  const int64_t nq = static_cast<int64_t>(pb->num_q_heads) * pb->head_dim;
  const int64_t nk = static_cast<int64_t>(pb->num_kv_heads) * pb->head_dim;
  const bool norm = gamma_q != nullptr;
  if ((dv_accum == nullptr) != (dv_in == nullptr))
    return fail(SEQATTN_ERR_INVALID_ARG, "dv_accum and dv_in must both be given or both be NULL");
  if ((s = check_ld(ld_dq, nq, "dq_in")) != SEQATTN_OK || (s = check_ld(ld_dk, nk, "dk_in")) != SEQATTN_OK) return s;
  if (dv_in != nullptr && (s = check_ld(ld_dv, nk, "dv_in")) != SEQATTN_OK) return s;
  if (norm && ((s = check_ld(ld_q, nq, "q_in")) != SEQATTN_OK || (s = check_ld(ld_k, nk, "k_in")) != SEQATTN_OK))
    return s;
  if (q_len == 0) return ok();
  s = check_ptrs({{dq, "dq"}, {dk_accum, "dk_accum"}, {dq_in, "dq_in"}, {dk_in, "dk_in"}});
  if (s != SEQATTN_OK) return s;
  if (!aligned16(dv_accum) || !aligned16(dv_in))
    return fail(SEQATTN_ERR_INVALID_ARG, "dv_accum or dv_in is not 16-byte aligned");
  s = check_apart({{dq_in, "dq_in"}, {dk_in, "dk_in"}, {dv_in, "dv_in"}},
                  {{dq, "dq"}, {dk_accum, "dk_accum"}, {dv_accum, "dv_accum"}});
  if (s != SEQATTN_OK) return s;
  if (norm) {
    s = check_ptrs({{q_in, "q_in"}, {k_in, "k_in"}, {dgamma_q, "dgamma_q"}, {dgamma_k, "dgamma_k"},
                    {workspace, "workspace"}});
    if (s != SEQATTN_OK) return s;
    if (workspace_size < norm_rope_workspace(pb->head_dim))
      return fail(SEQATTN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", workspace_size,
                  norm_rope_workspace(pb->head_dim));
    s = check_apart({{dq_in, "dq_in"}, {dk_in, "dk_in"}, {dv_in, "dv_in"}, {dgamma_q, "dgamma_q"},
                     {dgamma_k, "dgamma_k"}, {workspace, "workspace"}},
                    {{q_in, "q_in"}, {k_in, "k_in"}, {gamma_q, "gamma_q"}, {gamma_k, "gamma_k"}, {dq, "dq"},
                     {dk_accum, "dk_accum"}, {dv_accum, "dv_accum"}});
    if (s != SEQATTN_OK) return s;
    p.q_in = q_in;
    p.k_in = k_in;
    p.q_stride = ld_q;
    p.k_stride = ld_k;
    p.dgamma_q = dgamma_q;
    p.dgamma_k = dgamma_k;
    p.partial = static_cast<float*>(workspace);
  }
  p.dq = dq;
  p.dk = dk_accum;
  p.dv = dv_accum;
  p.dq_in = dq_in;
  p.dk_in = dk_in;
  p.dv_in = dv_in;
  p.dq_stride = ld_dq;
  p.dk_stride = ld_dk;
  p.dv_stride = ld_dv;
  const cudaError_t e = launch_norm_rope_bwd(p, pb->head_dim, pb->dtype == SEQATTN_BF16,
                                             reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "norm_rope_bwd launch");
}

static_assert(sizeof(seqattn_adamw_tensor) == sizeof(AdamwTensor), "the internal descriptor mirrors the public one");

seqattn_status seqattn_adamw_step(const seqattn_adamw_tensor* tensors, int32_t count, int32_t state_bits,
                                  const seqattn_adamw_params* params, seqattn_stream_t stream) {
  if (count < 0 || (count > 0 && tensors == nullptr) || params == nullptr)
    return fail(SEQATTN_ERR_INVALID_ARG, "tensors or params is NULL, or count (%d) < 0", count);
  if (state_bits != 8 && state_bits != 32)
    return fail(SEQATTN_ERR_INVALID_ARG, "state_bits %d is not 8 or 32", state_bits);
  const seqattn_adamw_params& a = *params;
  if (!(a.beta1 >= 0 && a.beta1 < 1 && a.beta2 >= 0 && a.beta2 < 1))
    return fail(SEQATTN_ERR_INVALID_ARG, "beta1 and beta2 must lie in [0, 1)");
  if (!isfinite(a.lr) || !isfinite(a.grad_scale) || !(a.eps >= 0 && isfinite(a.eps)))
    return fail(SEQATTN_ERR_INVALID_ARG, "lr and grad_scale must be finite, eps finite and >= 0");
  if (a.step < 1 && a.step_dev == nullptr)
    return fail(SEQATTN_ERR_INVALID_ARG, "step %lld < 1", (long long)a.step);
  if ((reinterpret_cast<uintptr_t>(a.lr_dev) & 3u) || (reinterpret_cast<uintptr_t>(a.grad_scale_dev) & 3u) ||
      (reinterpret_cast<uintptr_t>(a.step_dev) & 7u))
    return fail(SEQATTN_ERR_INVALID_ARG, "lr_dev, grad_scale_dev or step_dev is misaligned");
  for (int32_t i = 0; i < count; ++i) {
    const seqattn_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t{1} << 40))
      return fail(SEQATTN_ERR_INVALID_ARG, "tensor %d: n = %lld", i, (long long)t.n);
    if (!isfinite(t.weight_decay) || (t.grad_bf16 != 0 && t.grad_bf16 != 1))
      return fail(SEQATTN_ERR_INVALID_ARG, "tensor %d: weight_decay must be finite and grad_bf16 0 or 1", i);
    if (t.n == 0) continue;
    seqattn_status s = check_ptrs({{t.param, "param"}, {t.grad, "grad"}, {t.m, "m"}, {t.v, "v"}});
    if (s != SEQATTN_OK) return s;
    if (!aligned16(t.lowp)) return fail(SEQATTN_ERR_INVALID_ARG, "tensor %d: lowp is not 16-byte aligned", i);
    if (state_bits == 8 && (t.m_scale == nullptr || t.v_scale == nullptr ||
                            (reinterpret_cast<uintptr_t>(t.m_scale) & 3u) || (reinterpret_cast<uintptr_t>(t.v_scale) & 3u)))
      return fail(SEQATTN_ERR_INVALID_ARG, "tensor %d: m_scale or v_scale is NULL or not 4-byte aligned", i);
  }
  AdamwHyper h = {};
  h.lr = static_cast<float>(a.lr);
  h.beta1 = static_cast<float>(a.beta1);
  h.one_minus_beta1 = static_cast<float>(1.0 - a.beta1);
  h.beta2 = static_cast<float>(a.beta2);
  h.one_minus_beta2 = static_cast<float>(1.0 - a.beta2);
  h.eps = static_cast<float>(a.eps);
  h.grad_scale = static_cast<float>(a.grad_scale);
  if (a.step_dev == nullptr) {
    h.step_size = static_cast<float>(a.lr / (1.0 - pow(a.beta1, static_cast<double>(a.step))));
    h.inv_root_bc2 = 1.f / static_cast<float>(sqrt(1.0 - pow(a.beta2, static_cast<double>(a.step))));
  }
  h.lrd = a.lr;
  h.beta1d = a.beta1;
  h.beta2d = a.beta2;
  h.step = a.step;
  h.lr_dev = a.lr_dev;
  h.grad_scale_dev = a.grad_scale_dev;
  h.step_dev = a.step_dev;
  const cudaError_t e = launch_adamw(reinterpret_cast<const AdamwTensor*>(tensors), count, state_bits, h,
                                     reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "adamw launch");
}

}  // extern "C"
