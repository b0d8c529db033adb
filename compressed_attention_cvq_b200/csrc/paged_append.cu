// cvq_paged_append: new keys and values into the pages, keys and queries rotated on the way.
//
// One pass: every element is read once and written once, so memory bounds it (a long prompt)
// or the launch (a decode step).  A CTA takes a token, or some of its head rows where there are
// few tokens.  All its threads first load their rows' chunks (16 threads a row, 8 dims each, up
// to kRows rows a thread); under these loads two warps find the token's sequence and row and take
// the sine and cosine of a pair a lane; one barrier, and the rows are rotated and stored.  (A warp
// a token without a barrier measured 63 us on the 8192-token prompt, and every thread taking its
// own sines 51 us; this 46, 4.3 TB/s.)  A decode step of 32 tokens takes 2.6 us.
#include <algorithm>

#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kThreads = 256;
constexpr int kSlots = kThreads / 16;       // rows that a CTA takes at once
constexpr int kRows = 1;                    // rows in flight per thread: more CTAs instead measured best

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
__global__ void __launch_bounds__(kThreads, 6) paged_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float4 s_ph[kPairs / 2];                      // (cos, sin) of two pairs each
  __shared__ long long s_at;                               // element offset of the token's row of head 0; -1: none
  __shared__ bool s_live;
  const int i = blockIdx.x, c = threadIdx.x & 15, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = a.q != nullptr ? a.n_q_heads : 0, nk = nq + a.n_kv_heads, heads = nk + a.n_kv_heads;   // queries, keys, values
  const int stride = gridDim.y * kSlots;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Chunk<In> in[kRows];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * stride;
      if (r >= heads) continue;
      const In* src = r < nq ? static_cast<const In*>(a.q) + i * a.q_stride + r * kHeadDim
                    : r < nk ? static_cast<const In*>(a.k) + i * a.k_stride + (r - nq) * kHeadDim
                             : static_cast<const In*>(a.v) + i * a.v_stride + (r - nk) * kHeadDim;
      in[u] = *reinterpret_cast<const Chunk<In>*>(src + 8 * c);
    }
  };
  int r0 = blockIdx.y * kSlots + (threadIdx.x >> 4);
  load(r0);
  if (warp < kPairs / 32) {
    // the sequence: as many as end at or before i (offsets do not decrease); 32 probes at a time
    int b = 0, n = a.batch;
    while (n > 0) {
      const int step = (n + 31) / 32;
      const int ended = __popc(__ballot_sync(0xffffffffu, lane * step < n && a.tok_offsets[b + lane * step + 1] <= i));
      if (step == 1) {
        b += ended;
        break;
      }
      // it lies behind the last probe that has ended, and not behind the next
      const int from = ended == 0 ? 0 : (ended - 1) * step + 1, to = ended == 0 ? 0 : min(ended * step, n);
      b += from;
      n = to - from;
    }
    const bool live = b < a.batch;                         // else padding behind the last sequence
    long long at = -1;
    if (live) {
      const int p = a.seq_lens[b] - (a.tok_offsets[b + 1] - i);
      const long long pos = (a.pos_offsets != nullptr ? a.pos_offsets[b] : 0) + static_cast<long long>(p);
      int page = -1;
      if (p >= 0 && (p >> a.page_shift) < a.max_pages)
        page = a.page_table[static_cast<size_t>(b) * a.max_pages + (p >> a.page_shift)];
      const int j = threadIdx.x;
      reinterpret_cast<float2*>(s_ph)[j] = phase_exact(a.phase.F[j] * static_cast<unsigned long long>(pos));
      if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages))
        at = static_cast<long long>(page) * a.page_stride + static_cast<long long>(p & ((1 << a.page_shift) - 1)) * kHeadDim;
    }
    if (threadIdx.x == 0) {
      s_at = at;
      s_live = live;
      if (live && at < 0) atomicOr(a.fault, kFaultPage);
    }
  }
  __syncthreads();
  if (!s_live) return;
  const long long at = s_at;
  const float4 p0 = s_ph[2 * c], p1 = s_ph[2 * c + 1];
  const float co[4] = {p0.x, p0.z, p1.x, p1.z}, si[4] = {p0.y, p0.w, p1.y, p1.w};
  while (r0 < heads) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * stride;
      if (r >= heads) continue;
      float x[8];
#pragma unroll
      for (int d = 0; d < 8; ++d) x[d] = to_float(in[u].x[d]);
      if (r < nk) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float re = x[2 * v], im = x[2 * v + 1];
          x[2 * v] = re * co[v] - im * si[v];
          x[2 * v + 1] = re * si[v] + im * co[v];
        }
      }
      if (r < nq) {
        Chunk<In> out;
#pragma unroll
        for (int d = 0; d < 8; ++d) out.x[d] = from_float<In>(x[d]);
        *reinterpret_cast<Chunk<In>*>(static_cast<In*>(a.q_out) + (static_cast<size_t>(i) * nq + r) * kHeadDim + 8 * c) = out;
      } else if (at >= 0) {
        Kv* pool = static_cast<Kv*>(r < nk ? a.k_pages : a.v_pages);
        const int h = r < nk ? r - nq : r - nk;
        Chunk<Kv> out;
#pragma unroll
        for (int d = 0; d < 8; ++d) out.x[d] = from_float<Kv>(x[d]);
        *reinterpret_cast<Chunk<Kv>*>(pool + at + (static_cast<long long>(h) << a.page_shift) * kHeadDim + 8 * c) = out;
      }
    }
    r0 += kRows * stride;
    load(r0);
  }
}

template <typename In>
cudaError_t launch_in(const AppendArgs& a, int kv_dtype, cudaStream_t stream) {
  const int heads = (a.q != nullptr ? a.n_q_heads : 0) + 2 * a.n_kv_heads;
  // where there are fewer tokens than make 8 CTAs an SM of 148, several CTAs share a token's rows
  const int most = (heads + kSlots - 1) / kSlots;
  const dim3 grid(a.n_tokens, std::max(1, std::min(most, 8 * 148 / a.n_tokens)));
  return kv_dtype == CVQ_BF16 ? launch_chained(paged_append_kernel<In, __nv_bfloat16>, grid, kThreads, a, stream)
                              : launch_chained(paged_append_kernel<In, __half>, grid, kThreads, a, stream);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, int in_dtype, int kv_dtype, cudaStream_t stream) {
  if (in_dtype == CVQ_BF16) return launch_in<__nv_bfloat16>(a, kv_dtype, stream);
  if (in_dtype == CVQ_F16) return launch_in<__half>(a, kv_dtype, stream);
  return launch_in<float>(a, kv_dtype, stream);
}

}  // namespace cvq
