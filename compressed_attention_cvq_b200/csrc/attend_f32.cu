// Shared-prefix attention in fp32 on the CUDA cores: a tile of query rows that share a KV
// head against tiles of 64 cached tokens, one pass with the running maximum and sum of the
// softmax.  A tile is decoded from its codes and rotated once, then read by every row.
//
// Per tile and CTA: S = Q K^T as 16 x 16 threads of RPT rows x 4 tokens each, operands read
// from shared memory as float4 along the 128 dims (token rows padded to 132 floats: the 8
// lanes of a 16-byte phase then start 4 banks apart); the weights go through shared memory
// transposed so that O += P V reads RPT weights and 8 value dims per thread and token.
#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;          // tokens per tile
constexpr int kPad = kHeadDim + 4;

// key code and value code lookups of the two layouts
__device__ __forceinline__ int wide_code(const uint8_t* codes, const ServeArgs& a, int h, int G, int r, int t) {
  const size_t row = (static_cast<size_t>(h) * kWideGroups + G) * a.R + r;
  if (a.code_bits == 6) return packed6_code(codes + row * (static_cast<size_t>(a.t_cap) / 4 * 3), t);
  return codes[row * a.t_cap + t] & 63;
}

// 8 dims (chunk c) of the key and value of token t of KV head h, decoded from the codes; the
// key rotated by position t
__device__ __forceinline__ void decode_chunk(const ServeArgs& a, const unsigned long long* f_tab, int h, int t,
                                             int c, float (&k)[8], float (&v)[8]) {
#pragma unroll
  for (int d = 0; d < 8; ++d) k[d] = v[d] = 0.f;
  const float* kcb = a.key_cb + h * a.key_cb_stride;
  const float* vcb = a.val_cb + h * a.val_cb_stride;
  for (int r = 0; r < a.R; ++r) {
    size_t ko, vo;
    if (a.wide) {
      const int G = c >> 3;
      const size_t base = (static_cast<size_t>(G) * a.R + r) * kWideCodes;
      ko = (base + wide_code(a.key_codes, a, h, G, r, t)) * kWideGroupDim + 8 * (c & 7);
      vo = (base + wide_code(a.val_codes, a, h, G, r, t)) * kWideGroupDim + 8 * (c & 7);
    } else {
      const size_t row = ((static_cast<size_t>(h) * a.t_cap + t) * a.R + r) * kGroups + c;
      const size_t base = (static_cast<size_t>(c) * a.R + r) * kCodes;
      ko = (base + a.key_codes[row]) * kCodeword;
      vo = (base + a.val_codes[row]) * kVDims;
    }
    const float4 a0 = __ldg(reinterpret_cast<const float4*>(kcb + ko));
    const float4 a1 = __ldg(reinterpret_cast<const float4*>(kcb + ko) + 1);
    const float4 b0 = __ldg(reinterpret_cast<const float4*>(vcb + vo));
    const float4 b1 = __ldg(reinterpret_cast<const float4*>(vcb + vo) + 1);
    k[0] += a0.x; k[1] += a0.y; k[2] += a0.z; k[3] += a0.w;
    k[4] += a1.x; k[5] += a1.y; k[6] += a1.z; k[7] += a1.w;
    v[0] += b0.x; v[1] += b0.y; v[2] += b0.z; v[3] += b0.w;
    v[4] += b1.x; v[5] += b1.y; v[6] += b1.z; v[7] += b1.w;
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 ph = phase_exact(f_tab[4 * c + p] * static_cast<unsigned long long>(static_cast<unsigned>(t)));
    const float re = k[2 * p], im = k[2 * p + 1];
    k[2 * p] = re * ph.x - im * ph.y;
    k[2 * p + 1] = re * ph.y + im * ph.x;
  }
}

// RB query rows per CTA: the rows of a KV head are (sequence, head of the group) pairs, and
// blockIdx.z takes RB of them.
template <int RB>
__global__ void __launch_bounds__(kThreads) attend_f32_kernel(const __grid_constant__ ServeArgs a) {
  constexpr int RPT = RB / 16;
  extern __shared__ float4 smem4[];
  float* sq = reinterpret_cast<float*>(smem4);      // [RB][kPad]
  float* sk = sq + RB * kPad;                       // [kTile][kPad]
  float* sv = sk + kTile * kPad;                    // [kTile][128]
  float* sp = sk;                                   // [kTile][RB], over the keys once they are read
  __shared__ unsigned long long f_tab[kPairs];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");         // the merge
  const int split = blockIdx.x, h = blockIdx.y;
  const int rows = a.batch * a.group;
  const int r0 = blockIdx.z * RB;
  int L = a.lens[0];
  L = L < 0 ? 0 : (L > a.t_cap ? a.t_cap : L);
  const long long per = ((L + a.n_splits - 1LL) / a.n_splits + kTile - 1) / kTile * kTile;
  const int start = static_cast<int>(min(per * split, static_cast<long long>(L)));
  const int end = static_cast<int>(min(start + per, static_cast<long long>(L)));
  // global row (sequence, query head) of local row r
  auto grow = [&](int r) {
    const int rr = r0 + r;
    return static_cast<size_t>(rr / a.group) * a.n_q_heads + h * a.group + rr % a.group;
  };
  for (int i = tid; i < kPairs; i += kThreads) f_tab[i] = a.phase.F[i];
  for (int i = tid; i < RB * kHeadDim; i += kThreads) {
    const int r = i / kHeadDim, d = i % kHeadDim;
    float x = 0.f;
    if (r0 + r < rows && start < end) x = load_any(a.q, a.q_dtype, grow(r) * kHeadDim + d);
    sq[r * kPad + d] = x * (0.08838834764831845f * kLog2e);
  }
  float m[RPT], l[RPT], o[RPT][8];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d) o[i][d] = 0.f;
  }
  for (int t0 = start; t0 < end; t0 += kTile) {
    __syncthreads();                                // the last tile's readers are done
#pragma unroll
    for (int u = 0; u < kTile * 16 / kThreads; ++u) {
      const int i = tid + u * kThreads, tk = i >> 4, c = i & 15, t = t0 + tk;
      float k[8], v[8];
      if (t < end) {
        decode_chunk(a, f_tab, h, t, c, k, v);
      } else {
#pragma unroll
        for (int d = 0; d < 8; ++d) k[d] = v[d] = 0.f;
      }
      float4* kd = reinterpret_cast<float4*>(sk + tk * kPad + 8 * c);
      kd[0] = make_float4(k[0], k[1], k[2], k[3]);
      kd[1] = make_float4(k[4], k[5], k[6], k[7]);
      float4* vd = reinterpret_cast<float4*>(sv + tk * kHeadDim + 8 * c);
      vd[0] = make_float4(v[0], v[1], v[2], v[3]);
      vd[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __syncthreads();
    float s[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int d = 0; d < kHeadDim; d += 4) {
      float4 qv[RPT], kv[4];
#pragma unroll
      for (int i = 0; i < RPT; ++i) qv[i] = *reinterpret_cast<const float4*>(sq + (ty * RPT + i) * kPad + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * kPad + d);
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
          s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
          s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
          s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
        }
    }
    __syncthreads();                                // sp takes the place of sk
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (t0 + tx + 16 * j >= end) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) s[i][j] = -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;          // nothing seen yet: every weight 0
      const float alpha = exp2f(m[i] - ref);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - ref);
        sum += p;
        sp[(tx + 16 * j) * RB + ty * RPT + i] = p;
      }
      l[i] = fmaf(l[i], alpha, sum);
#pragma unroll
      for (int d = 0; d < 8; ++d) o[i][d] *= alpha;
    }
    __syncthreads();
    for (int t = 0; t < kTile; ++t) {
      float p[RPT];
      if constexpr (RPT == 4) {
        const float4 pv = *reinterpret_cast<const float4*>(sp + t * RB + ty * RPT);
        p[0] = pv.x; p[1] = pv.y; p[2] = pv.z; p[3] = pv.w;
      } else {
#pragma unroll
        for (int i = 0; i < RPT; ++i) p[i] = sp[t * RB + ty * RPT + i];
      }
      const float4 v0 = *reinterpret_cast<const float4*>(sv + t * kHeadDim + 4 * tx);
      const float4 v1 = *reinterpret_cast<const float4*>(sv + t * kHeadDim + 64 + 4 * tx);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        o[i][0] = fmaf(p[i], v0.x, o[i][0]);
        o[i][1] = fmaf(p[i], v0.y, o[i][1]);
        o[i][2] = fmaf(p[i], v0.z, o[i][2]);
        o[i][3] = fmaf(p[i], v0.w, o[i][3]);
        o[i][4] = fmaf(p[i], v1.x, o[i][4]);
        o[i][5] = fmaf(p[i], v1.y, o[i][5]);
        o[i][6] = fmaf(p[i], v1.z, o[i][6]);
        o[i][7] = fmaf(p[i], v1.w, o[i][7]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int r = ty * RPT + i;
    if (r0 + r >= rows) continue;
    const size_t at = grow(r) * a.n_parts + split;
    if (tx == 0) {
      a.part_m[at] = m[i];
      a.part_l[at] = l[i];
    }
    if (start >= end) continue;
    float4* po = reinterpret_cast<float4*>(a.part_o + at * kHeadDim);
    po[tx] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    po[16 + tx] = make_float4(o[i][4], o[i][5], o[i][6], o[i][7]);
  }
}

// Merge of the partial states of a row (m in log2 units): a CTA per (sequence, query head), the
// states strided over its warps, 4 dims a lane and U states in flight; the warps' sums are joined
// in their order.  It is launched while the attention kernel still runs and waits for its end.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const __grid_constant__ ServeArgs a) {
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ float4 s_o[kMergeWarps][32];
  const size_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* pm = a.part_m + row * a.n_parts;
  const float* pl = a.part_l + row * a.n_parts;
  const float4* po = reinterpret_cast<const float4*>(a.part_o + row * a.n_parts * kHeadDim) + lane;
  constexpr int U = 8;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int s0 = warp; s0 < a.n_parts; s0 += U * kMergeWarps) {
    float mv[U], lv[U];
    float4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * kMergeWarps;
      const bool in = s < a.n_parts;
      mv[u] = in ? __ldcg(pm + s) : -INFINITY;
      lv[u] = in ? __ldcg(pl + s) : 0.f;
      x[u] = in ? __ldcg(po + static_cast<size_t>(s) * (kHeadDim / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mn = M;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = fmaxf(mn, mv[u]);
    const float alpha = mn == -INFINITY ? 1.f : exp2f(M - mn);
    M = mn;
    L *= alpha;
    acc = make_float4(acc.x * alpha, acc.y * alpha, acc.z * alpha, acc.w * alpha);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (mv[u] == -INFINITY && lv[u] == 0.f) continue;       // a part with no token has no o
      const float f = exp2f(mv[u] - M);
      L = fmaf(lv[u], f, L);
      acc = make_float4(fmaf(x[u].x, f, acc.x), fmaf(x[u].y, f, acc.y), fmaf(x[u].z, f, acc.z), fmaf(x[u].w, f, acc.w));
    }
  }
  s_o[warp][lane] = acc;
  if (lane == 0) {
    s_m[warp] = M;
    s_l[warp] = L;
  }
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) M = fmaxf(M, s_m[w]);
  L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    if (s_m[w] == -INFINITY && s_l[w] == 0.f) continue;
    const float f = exp2f(s_m[w] - M);
    const float4 x = s_o[w][lane];
    L = fmaf(s_l[w], f, L);
    acc = make_float4(fmaf(x.x, f, acc.x), fmaf(x.y, f, acc.y), fmaf(x.z, f, acc.z), fmaf(x.w, f, acc.w));
  }
  const float4 y = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x / L, acc.y / L, acc.z / L, acc.w / L);
  store_four(a.out, a.out_dtype, row * kHeadDim + 4 * lane, y);
  if (lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int RB>
cudaError_t run(const ServeArgs& a, dim3 grid, cudaStream_t stream) {
  static PerDeviceFlag flag;
  const size_t bytes = (static_cast<size_t>(RB) * kPad + kTile * kPad + kTile * kHeadDim) * sizeof(float);
  static_assert(RB <= kPad, "the weights fit over the keys");
  const cudaError_t e = set_smem_limit_once(flag, attend_f32_kernel<RB>, bytes);
  if (e != cudaSuccess) return e;
  attend_f32_kernel<RB><<<grid, kThreads, bytes, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_f32(const ServeArgs& a, cudaStream_t stream) {
  const int rows = a.batch * a.group;
  const dim3 grid(a.n_splits, a.n_kv_heads, rows <= 16 ? 1 : (rows + 63) / 64);
  return rows <= 16 ? run<16>(a, grid, stream) : run<64>(a, grid, stream);
}

cudaError_t launch_merge(const ServeArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * a.n_q_heads);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel, a);
}

}  // namespace cvq
