// cvq_paged_append: new keys and values into the pages, keys and queries rotated on the way.
//
// One pass: every element is read once and written once, so memory bounds it (a long prompt)
// or the launch (a decode step).  A CTA takes one token; 16 threads share a head row as
// 16-byte (16-bit input) or 32-byte (fp32) chunks of 8 dims, and a thread keeps its chunk of
// 4 RoPE pairs while it walks the heads, so that the sines of a token are taken once per
// CTA slice and not once per head.
#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kThreads = 256;
constexpr int kSlots = kThreads / 16;       // heads in flight per CTA

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }

template <typename T>
struct alignas(16) Chunk {
  T x[8];
};

template <typename In, typename Kv>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ AppendArgs a) {
  const int i = blockIdx.x;                                // the token
  const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
  // the sequence: as many as end at or before i (offsets do not decrease)
  int before = 0;
  for (int j0 = 0; j0 < a.batch; j0 += kThreads) {
    const int j = j0 + static_cast<int>(threadIdx.x);
    before += __syncthreads_count(j < a.batch && a.tok_offsets[j + 1] <= i);
  }
  const int b = before;
  if (b >= a.batch) return;                                // padding behind the last sequence
  const int p = a.seq_lens[b] - (a.tok_offsets[b + 1] - i);
  const long long pos = (a.pos_offsets != nullptr ? a.pos_offsets[b] : 0) + static_cast<long long>(p);
  long long at = -1;                                       // element offset of the token's row of head 0
  if (p >= 0 && (p >> a.page_shift) < a.max_pages) {
    const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + (p >> a.page_shift)];
    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages))
      at = static_cast<long long>(page) * a.page_stride + static_cast<long long>(p & ((1 << a.page_shift) - 1)) * kHeadDim;
  }
  if (at < 0 && threadIdx.x == 0) atomicOr(a.fault, kFaultPage);
  float2 ph[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    ph[u] = phase_exact(a.phase.F[4 * c + u] * static_cast<unsigned long long>(pos));
  const int nq = a.q != nullptr ? a.n_q_heads : 0;
  const int heads = nq + 2 * a.n_kv_heads;                 // queries, keys, values
  for (int hd = blockIdx.y * kSlots + slot; hd < heads; hd += gridDim.y * kSlots) {
    const In* src;
    if (hd < nq) src = static_cast<const In*>(a.q) + i * a.q_stride + hd * kHeadDim;
    else if (hd < nq + a.n_kv_heads) src = static_cast<const In*>(a.k) + i * a.k_stride + (hd - nq) * kHeadDim;
    else src = static_cast<const In*>(a.v) + i * a.v_stride + (hd - nq - a.n_kv_heads) * kHeadDim;
    if (hd >= nq && at < 0) continue;
    const Chunk<In> in = *reinterpret_cast<const Chunk<In>*>(src + 8 * c);
    float x[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) x[d] = to_float(in.x[d]);
    if (hd < nq + a.n_kv_heads) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float re = x[2 * u], im = x[2 * u + 1];
        x[2 * u] = re * ph[u].x - im * ph[u].y;
        x[2 * u + 1] = re * ph[u].y + im * ph[u].x;
      }
    }
    if (hd < nq) {
      Chunk<In> out;
#pragma unroll
      for (int d = 0; d < 8; ++d) out.x[d] = from_float<In>(x[d]);
      *reinterpret_cast<Chunk<In>*>(static_cast<In*>(a.q_out) + (static_cast<size_t>(i) * nq + hd) * kHeadDim + 8 * c) = out;
    } else {
      const bool key = hd < nq + a.n_kv_heads;
      const int h = key ? hd - nq : hd - nq - a.n_kv_heads;
      Kv* pool = static_cast<Kv*>(key ? a.k_pages : a.v_pages);
      Chunk<Kv> out;
#pragma unroll
      for (int d = 0; d < 8; ++d) out.x[d] = from_float<Kv>(x[d]);
      *reinterpret_cast<Chunk<Kv>*>(pool + at + (static_cast<long long>(h) << a.page_shift) * kHeadDim + 8 * c) = out;
    }
  }
}

template <typename In>
cudaError_t launch_in(const AppendArgs& a, int kv_dtype, cudaStream_t stream) {
  const int heads = (a.q != nullptr ? a.n_q_heads : 0) + 2 * a.n_kv_heads;
  const dim3 grid(a.n_tokens, a.n_tokens >= 1024 ? 1 : (heads + kSlots - 1) / kSlots);
  if (kv_dtype == CVQ_BF16) paged_append_kernel<In, __nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  else paged_append_kernel<In, __half><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, int in_dtype, int kv_dtype, cudaStream_t stream) {
  if (in_dtype == CVQ_BF16) return launch_in<__nv_bfloat16>(a, kv_dtype, stream);
  if (in_dtype == CVQ_F16) return launch_in<__half>(a, kv_dtype, stream);
  return launch_in<float>(a, kv_dtype, stream);
}

}  // namespace cvq
