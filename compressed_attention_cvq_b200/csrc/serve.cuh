// Shared definitions of the serving operators: shared-prefix attention, the paged 16-bit
// cache and the attention over it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace cvq {

constexpr unsigned int kFaultPage = CVQ_PAGE_FAULT;

// A workspace starts with the arrival counters of paged calls, one per (sequence, KV head), at a
// place that no call's states reach, whatever its shape: so every paged call finds them as the last one
// left them, at zero.  Calls of more units than that have CTAs enough without splits.
constexpr int kCounters = 16384;
constexpr size_t kCounterBytes = kCounters * sizeof(int);

// Arguments of the attention kernels.  Split partial states are [B, Hq, n_splits] rows as in
// the other decode kernels, with m in log2 units (the kernels work with exp2); a split with
// no token stores m = -inf and l = 0 and leaves its o unwritten.
struct ServeArgs {
  const void* q;
  int q_dtype;
  int batch, n_q_heads, n_kv_heads, group;
  int n_splits;
  int n_parts;                    // partial states per row: n_splits, or one per CTA of their clusters
  float* part_o;
  float* part_m;
  float* part_l;
  int* counters;
  const int32_t* lens;            // prefix_len [1] or seq_lens [B]
  int t_cap;                      // tokens the cache (or a table row) can hold
  unsigned int* fault;
  const float* prev_out;
  const float* prev_lse;
  void* out;
  int out_dtype;
  float* lse;
  // code cache (prefix)
  const float* key_cb;
  const float* val_cb;
  long long key_cb_stride, val_cb_stride;
  const uint8_t* key_codes;
  const uint8_t* val_codes;
  int R, wide, code_bits;
  PhaseTurns phase;
  void* book;                     // codebooks in the tensor-core kernel's order
  uint32_t* book_peak;            // their largest elements
  float* kept_o;                  // [row][part][2][128], sums of long streams
  // paged cache
  const void* k_pages;
  const void* v_pages;
  const int32_t* page_table;
  int kv_dtype, page_shift, n_pages, max_pages;
  long long page_stride;
};

struct AppendArgs {
  const void* q;
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;
  const int32_t* tok_offsets;
  const int32_t* seq_lens;
  const int32_t* pos_offsets;
  const int32_t* page_table;
  void* k_pages;
  void* v_pages;
  void* q_out;
  int n_tokens, batch, n_q_heads, n_kv_heads, page_shift, n_pages, max_pages;
  long long page_stride;
  unsigned int* fault;
  PhaseTurns phase;
};

// The tensor-core kernel: tokens of a CTA's tile, and its tiles of a stream (every other one of a CTA)
// between flushes of its O.  Outputs are 3e-6 off at most (32: 7e-6, and 260 us at 131072 tokens where 16
// takes 271).
constexpr int kTok = 64;
constexpr int kFlush = 16;

// partial states of a call, and rows of its outputs
__device__ __forceinline__ size_t n_part_rows(const ServeArgs& a) { return static_cast<size_t>(a.batch) * a.n_q_heads * a.n_parts; }
__device__ __forceinline__ size_t n_rows(const ServeArgs& a) { return static_cast<size_t>(a.batch) * a.n_q_heads; }

__device__ __forceinline__ float load_any(const void* p, int dtype, size_t i) {
  if (dtype == CVQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == CVQ_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// four elements from i on (a multiple of 4)
__device__ __forceinline__ void store_four(void* p, int dtype, size_t i, float4 x) {
  if (dtype == CVQ_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = x;
  } else if (dtype == CVQ_BF16) {
    __nv_bfloat162* at = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p) + i);
    at[0] = __floats2bfloat162_rn(x.x, x.y);
    at[1] = __floats2bfloat162_rn(x.z, x.w);
  } else {
    __half2* at = reinterpret_cast<__half2*>(static_cast<__half*>(p) + i);
    at[0] = __floats2half2_rn(x.x, x.y);
    at[1] = __floats2half2_rn(x.z, x.w);
  }
}

// e^{2 pi i turn64 / 2^64} to full fp32 accuracy (phase_from_turn's __sincosf is good to
// 2^-21; here outputs may be fp32): the signed top 32 bits are the angle in units of
// 2^-31 pi, rounded once to fp32.
__device__ __forceinline__ float2 phase_exact(unsigned long long turn64) {
  const float x = static_cast<float>(static_cast<int>(turn64 >> 32)) * 4.656612873077393e-10f;
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c, s);
}

// A launch that may begin while the kernel before it in the stream ends; the kernel waits
// (griddepcontrol.wait) before it touches memory.
template <typename Args>
cudaError_t launch_chained(void (*kernel)(const Args), dim3 grid, int threads, const Args& a, cudaStream_t stream, size_t smem = 0) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// the checks of cvq_shape and of a codebook head stride (api.cu)
cvq_status check_shape_status(const cvq_shape* s);
cvq_status check_codebook_stride(const cvq_shape* s, int64_t stride);

cudaError_t launch_prefix_f32(const ServeArgs& a, cudaStream_t stream);
cudaError_t launch_prefix_mma(const ServeArgs& a, cudaStream_t stream);   // 16-bit queries
cudaError_t launch_paged_attend(const ServeArgs& a, cudaStream_t stream);
cudaError_t launch_merge(const ServeArgs& a, cudaStream_t stream);
cudaError_t launch_paged_append(const AppendArgs& a, int in_dtype, int kv_dtype, cudaStream_t stream);

}  // namespace cvq
