// cvq_paged_append: new keys and values into the pages, keys and queries rotated on the way.
//
// One pass: every element is read once and written once, so memory bounds it (a long prompt)
// or the launch (a decode step).  A CTA takes a token, or some of its head rows where there are
// few tokens.  All its threads first load their chunk of a row (16 bytes: 8 dims of 16-bit input, 4 of
// fp32); under these loads two warps find the token's sequence and row and take
// the sine and cosine of a pair a lane; one barrier, and the rows are rotated and stored.  Many
// small CTAs with two chunks a thread in flight measured best: 8192 tokens of 32 + 16 heads in bf16 take
// 40 us (5.1 TB/s; a copy of the same bytes by the framework 67), with one chunk 42, with 256 threads
// more, a warp a token without a barrier 63; 1531 tokens of fp32 8.7 us (some of it from L2; 12.3 from
// memory), a decode step of 32 tokens 2.5 us.
#include <algorithm>

#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kThreads = 128;

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

template <typename T, int N>
struct alignas(N * sizeof(T)) Chunk {
  T x[N];
};

template <typename In>
constexpr int kDims = 16 / sizeof(In);

template <typename In, typename Kv>
__global__ void __launch_bounds__(kThreads, 12) paged_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kD = kDims<In>, kLanes = kHeadDim / kD, kSlots = kThreads / kLanes;   // kSlots rows at once
  __shared__ float4 s_ph[kPairs / 2];                      // (cos, sin) of two pairs each
  __shared__ long long s_at;                               // element offset of the token's row of head 0; -1: none
  __shared__ bool s_live;
  const int i = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = threadIdx.x % kLanes;
  const int nq = a.q != nullptr ? a.n_q_heads : 0, nk = nq + a.n_kv_heads, heads = nk + a.n_kv_heads;   // queries, keys, values
  const int stride = gridDim.y * kSlots;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Chunk<In, kD> in;
  auto load = [&](int r, Chunk<In, kD>& in) {
    if (r < heads) {
      const In* src = r < nq ? static_cast<const In*>(a.q) + i * a.q_stride + r * kHeadDim
                    : r < nk ? static_cast<const In*>(a.k) + i * a.k_stride + (r - nq) * kHeadDim
                             : static_cast<const In*>(a.v) + i * a.v_stride + (r - nk) * kHeadDim;
      in = *reinterpret_cast<const Chunk<In, kD>*>(src + kD * c);
    }
  };
  int r = blockIdx.y * kSlots + threadIdx.x / kLanes;
  load(r, in);
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
      if (p >= 0 && (p >> a.page_shift) < a.max_pages && in_bounds(a.fault, b, a.batch))
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
  float4 ph[kD / 4];                                       // (cos, sin) of two pairs each
#pragma unroll
  for (int v = 0; v < kD / 4; ++v) ph[v] = s_ph[c * (kD / 4) + v];
  while (r < heads) {
    Chunk<In, kD> next;                                    // under this one's arithmetic
    load(r + stride, next);
    float x[kD];
#pragma unroll
    for (int d = 0; d < kD; ++d) x[d] = to_float(in.x[d]);
    if (r < nk) {
#pragma unroll
      for (int v = 0; v < kD / 2; ++v) {
        const float re = x[2 * v], im = x[2 * v + 1];
        const float co = v % 2 == 0 ? ph[v / 2].x : ph[v / 2].z, si = v % 2 == 0 ? ph[v / 2].y : ph[v / 2].w;
        x[2 * v] = re * co - im * si;
        x[2 * v + 1] = re * si + im * co;
      }
    }
    if (r < nq) {
      Chunk<In, kD> out;
#pragma unroll
      for (int d = 0; d < kD; ++d) out.x[d] = from_float<In>(x[d]);
      if (in_bounds(a.fault, r, a.n_q_heads) && in_bounds(a.fault, i, a.n_tokens))
        *reinterpret_cast<Chunk<In, kD>*>(static_cast<In*>(a.q_out) + (static_cast<size_t>(i) * nq + r) * kHeadDim + kD * c) = out;
    } else if (at >= 0) {
      Kv* pool = static_cast<Kv*>(r < nk ? a.k_pages : a.v_pages);
      const int h = r < nk ? r - nq : r - nk;
      Chunk<Kv, kD> out;
#pragma unroll
      for (int d = 0; d < kD; ++d) out.x[d] = from_float<Kv>(x[d]);
      if (in_bounds(a.fault, h, a.n_kv_heads) && in_bounds(a.fault, at, a.n_pages * a.page_stride))
        *reinterpret_cast<Chunk<Kv, kD>*>(pool + at + (static_cast<long long>(h) << a.page_shift) * kHeadDim + kD * c) = out;
    }
    r += stride;
    in = next;
  }
}

template <typename In>
cudaError_t launch_in(const AppendArgs& a, int kv_dtype, cudaStream_t stream) {
  const int heads = (a.q != nullptr ? a.n_q_heads : 0) + 2 * a.n_kv_heads;
  // where there are fewer tokens than make 12 CTAs an SM of 148, several CTAs share a token's rows
  constexpr int kSlots = kThreads / (kHeadDim / kDims<In>);
  const int most = (heads + kSlots - 1) / kSlots;
  const dim3 grid(a.n_tokens, std::max(1, std::min(most, 12 * 148 / a.n_tokens)));
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
