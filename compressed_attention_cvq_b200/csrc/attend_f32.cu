// Shared-prefix attention in fp32 on the CUDA cores: a tile of query rows that share a KV
// head against tiles of 64 cached tokens, one pass with the running maximum and sum of the
// softmax.  A tile is decoded from its codes and rotated once, then read by every row.
//
// Per tile and CTA: S = Q K^T as 16 x 16 threads of RPT rows x 4 tokens each, operands read
// from shared memory as float4 along the 128 dims (token rows padded to 132 floats: the 8
// lanes of a 16-byte phase then start 4 banks apart); the weights go through shared memory
// transposed so that O += P V reads RPT weights and 8 value dims per thread and token.
//
// What bounds it: shared-memory operands (for 64 rows 8 float4 loads per 64 FMA, for up to 16 rows,
// where a thread has two, 6 per 32) and, for one tile per CTA, its chain of two gathers.  4 sequences
// over 1000 tokens, R = 1, 10.9 us with the merge; 16 over 8192 95 us.
#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;          // tokens per tile
constexpr int kPad = kHeadDim + 4;

// key code and value code lookups of the two layouts
__device__ __forceinline__ int wide_code(const uint8_t* codes, const ServeArgs& a, int h, int G, int r, int t) {
  const size_t row = (static_cast<size_t>(h) * kWideGroups + G) * a.R + r;
  if (!in_bounds(a.fault, t, a.t_cap)) return 0;
  if (a.code_bits == 6) return packed6_code(codes + row * (static_cast<size_t>(a.t_cap) / 4 * 3), t);
  return codes[row * a.t_cap + t] & 63;
}

__device__ __forceinline__ void add8(float (&x)[8], const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] += a.x; x[1] += a.y; x[2] += a.z; x[3] += a.w;
  x[4] += b.x; x[5] += b.y; x[6] += b.z; x[7] += b.w;
}
__device__ __forceinline__ void put8(float* at, const float (&x)[8]) {
  reinterpret_cast<float4*>(at)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(at)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// One side of a tile: 8 dims (chunk c = tid % 16) of kPer tokens a thread, all of whose codes are
// loaded before the first codeword and all of whose codewords before the first sum (8-scalar
// groups, kR rounds; 64-scalar groups, kR = 0, go round by round).
constexpr int kPer = kTile * 16 / kThreads, kStep = kThreads / 16;
template <int kR>
__device__ __forceinline__ void decode_side(const ServeArgs& a, const float* cb, const uint8_t* codes, int h, int t0, int end,
                                            float (&x)[kPer][8]) {
  const int c = threadIdx.x & 15, tk = threadIdx.x >> 4;
#pragma unroll
  for (int u = 0; u < kPer; ++u)
#pragma unroll
    for (int d = 0; d < 8; ++d) x[u][d] = 0.f;
  if constexpr (kR > 0) {
    int code[kPer * kR];
#pragma unroll
    for (int j = 0; j < kPer * kR; ++j) {
      const int t = t0 + min(tk + j / kR * kStep, end - 1 - t0);       // t0 + 64 may pass 32 bits
      code[j] = in_bounds(a.fault, t, a.t_cap) ? __ldg(codes + ((static_cast<size_t>(h) * a.t_cap + t) * kR + j % kR) * kGroups + c) : 0;
    }
#pragma unroll
    for (int j = 0; j < kPer * kR; ++j) add8(x[j / kR], cb + ((static_cast<size_t>(c) * kR + j % kR) * kCodes + code[j]) * kCodeword);
  } else {
    const int G = c >> 3;
    for (int r = 0; r < a.R; ++r) {
      const float* book = cb + (static_cast<size_t>(G) * a.R + r) * (kWideCodes * kWideGroupDim) + 8 * (c & 7);
#pragma unroll
      for (int u = 0; u < kPer; ++u)
        add8(x[u], book + wide_code(codes, a, h, G, r, t0 + min(tk + u * kStep, end - 1 - t0)) * kWideGroupDim);
    }
  }
}

// A tile of keys and values, decoded, the keys rotated by their positions; tokens from `end` on
// are zeros.
template <int kR>
__device__ __forceinline__ void make_tile(const ServeArgs& a, const unsigned long long* f_tab, int h, int t0, int end,
                                          float* sk, float* sv) {
  const int c = threadIdx.x & 15, tk = threadIdx.x >> 4;
  float x[kPer][8];
  decode_side<kR>(a, a.key_cb + h * a.key_cb_stride, a.key_codes, h, t0, end, x);
  // phases of the first token, turned on to the others (one fp32 rounding each)
  float2 ph[4], step[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    ph[p] = phase_exact(f_tab[4 * c + p] * static_cast<unsigned long long>(static_cast<unsigned>(t0) + tk));
    step[p] = phase_exact(f_tab[4 * c + p] * kStep);
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int row = tk + u * kStep;
    if (u > 0) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
        ph[p] = make_float2(ph[p].x * step[p].x - ph[p].y * step[p].y, ph[p].x * step[p].y + ph[p].y * step[p].x);
    }
    const bool in = row < end - t0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float re = x[u][2 * p], im = x[u][2 * p + 1];
      x[u][2 * p] = in ? re * ph[p].x - im * ph[p].y : 0.f;
      x[u][2 * p + 1] = in ? re * ph[p].y + im * ph[p].x : 0.f;
    }
    put8(sk + row * kPad + 8 * c, x[u]);
  }
  decode_side<kR>(a, a.val_cb + h * a.val_cb_stride, a.val_codes, h, t0, end, x);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int row = tk + u * kStep;
    if (row >= end - t0) {
#pragma unroll
      for (int d = 0; d < 8; ++d) x[u][d] = 0.f;
    }
    put8(sv + row * kHeadDim + 8 * c, x[u]);
  }
}

// RB query rows per CTA: the rows of a KV head are (sequence, head of the group) pairs, and
// blockIdx.z takes RB of them.
// Two CTAs an SM where they have room for it, but one of 64 rows and 8-scalar groups: a second one's
// tiles would take the L1 cache that its codewords are gathered through (R = 2: 110 us against 125;
// 64-scalar groups 119 against 101).
template <int RB, bool kWide>
__global__ void __launch_bounds__(kThreads, RB == 16 || kWide ? 2 : 1) attend_f32_kernel(const __grid_constant__ ServeArgs a) {
  // few rows: the threads are two halves, which share the dims of the scores and the tokens of the
  // outputs, so that a thread has two rows and reads fewer operands per product
  constexpr int kHalves = RB == 16 ? 2 : 1, RPT = RB * kHalves / 16;
  extern __shared__ float4 smem4[];
  float* sq = reinterpret_cast<float*>(smem4);      // [RB][kPad]
  float* sk = sq + RB * kPad;                       // [kTile][kPad]
  float* sv = sk + kTile * kPad;                    // [kTile][128]
  float* sp = sk;                                   // [kTile][RB], over the keys once they are read
  float* sum = sk + kTile * RB;                     // [2][RB][kTile], two halves' scores, also over the keys
  static_assert(kHalves == 1 || kTile * RB + 2 * RB * kTile <= kTile * kPad, "they fit");
  __shared__ unsigned long long f_tab[kPairs];
  const int tid = threadIdx.x, tx = tid & 15, half = kHalves == 2 ? tid >> 7 : 0, ty = (tid >> 4) & (16 / kHalves - 1);
  asm volatile("griddepcontrol.wait;" ::: "memory");                        // for what ran before this call
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");         // the merge
  const int split = blockIdx.x, h = blockIdx.y;
  const int rows = a.batch * a.group;
  const int r0 = blockIdx.z * RB;
  int L = a.lens[0];
  L = L < 0 ? 0 : (L > a.t_cap ? a.t_cap : L);
  const long long per = ((static_cast<long long>(L) + a.n_splits - 1) / a.n_splits + kTile - 1) / kTile * kTile;
  const int start = static_cast<int>(min(per * split, static_cast<long long>(L)));
  const int end = static_cast<int>(min(start + per, static_cast<long long>(L)));
  // global row (sequence, query head) of local row r
  auto grow = [&](int r) {
    const int rr = r0 + r;
    return static_cast<size_t>(rr / a.group) * a.n_q_heads + h * a.group + rr % a.group;
  };
  for (int i = tid; i < kPairs; i += kThreads) f_tab[i] = a.phase.F[i];
  // 8 elements of a query row, scaled; few rows are loaded here and stored under the first tile's
  // gathers
  auto query = [&](int i, float (&x)[8]) {
    const int r = i / 16;
    if (r0 + r >= rows || start >= end || !in_bounds(a.fault, grow(r), n_rows(a))) {
#pragma unroll
      for (int d = 0; d < 8; ++d) x[d] = 0.f;
      return;
    }
    const size_t at = grow(r) * kHeadDim + i % 16 * 8;
    if (a.q_dtype == CVQ_F32) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at) + 1);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
      x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
#pragma unroll
      for (int d = 0; d < 8; ++d) x[d] = load_any(a.q, a.q_dtype, at + d);
    }
  };
  auto put_query = [&](int i, float (&x)[8]) {
#pragma unroll
    for (int d = 0; d < 8; ++d) x[d] *= 0.08838834764831845f * kLog2e;
    put8(sq + i / 16 * kPad + i % 16 * 8, x);
  };
  float early[8];
  if (RB == 16) {
    query(tid, early);
  } else {
#pragma unroll 1
    for (int i = tid; i < RB * 16; i += kThreads) {
      query(i, early);
      put_query(i, early);
    }
  }
  __syncthreads();                                  // f_tab
  float m[RPT], l[RPT], o[RPT][8];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d) o[i][d] = 0.f;
  }
  const int ntiles = static_cast<int>((static_cast<long long>(end) - start + kTile - 1) / kTile);
  for (int i = 0; i < ntiles; ++i) {
    const int t0 = start + i * kTile;
    __syncthreads();                                // the last tile's readers are done
    if constexpr (kWide) make_tile<0>(a, f_tab, h, t0, end, sk, sv);
    else if (a.R == 1) make_tile<1>(a, f_tab, h, t0, end, sk, sv);
    else make_tile<2>(a, f_tab, h, t0, end, sk, sv);
    if (RB == 16 && i == 0) put_query(tid, early);
    __syncthreads();
    float s[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = half * (kHeadDim / kHalves); d < (half + 1) * (kHeadDim / kHalves); d += 4) {
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
    if constexpr (kHalves == 2) {
      auto at = [&](int w, int i, int j) -> float& { return sum[(w * RB + ty * RPT + i) * kTile + tx + 16 * j]; };
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) at(half, i, j) = s[i][j];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] += at(1 - half, i, j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (tx + 16 * j >= end - t0) {
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
      float total = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - ref);
        total += p;
        if (half == 0) sp[(tx + 16 * j) * RB + ty * RPT + i] = p;
      }
      l[i] = fmaf(l[i], alpha, total);
#pragma unroll
      for (int d = 0; d < 8; ++d) o[i][d] *= alpha;
    }
    __syncthreads();
#pragma unroll 8
    for (int t = half * (kTile / kHalves); t < (half + 1) * (kTile / kHalves); ++t) {
      float p[RPT];
      if constexpr (RPT == 4) {
        const float4 pv = *reinterpret_cast<const float4*>(sp + t * RB + ty * RPT);
        p[0] = pv.x; p[1] = pv.y; p[2] = pv.z; p[3] = pv.w;
      } else {
        static_assert(RPT == 2 || RPT == 4, "rows of a thread");
        const float2 pv = *reinterpret_cast<const float2*>(sp + t * RB + ty * RPT);
        p[0] = pv.x; p[1] = pv.y;
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
  if constexpr (kHalves == 2) {
    __syncthreads();                                // the weights have been read
    float4* other = reinterpret_cast<float4*>(sk) + (ty * RPT) * (kHeadDim / 4) + tx;
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        other[i * (kHeadDim / 4)] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        other[i * (kHeadDim / 4) + 16] = make_float4(o[i][4], o[i][5], o[i][6], o[i][7]);
      }
    }
    __syncthreads();
    if (half == 1) return;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float4 u = other[i * (kHeadDim / 4)], v = other[i * (kHeadDim / 4) + 16];
      o[i][0] += u.x; o[i][1] += u.y; o[i][2] += u.z; o[i][3] += u.w;
      o[i][4] += v.x; o[i][5] += v.y; o[i][6] += v.z; o[i][7] += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int r = ty * RPT + i;
    if (r0 + r >= rows) continue;
    const size_t at = grow(r) * a.n_parts + split;
    if (!in_bounds(a.fault, at, n_part_rows(a))) continue;
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
      const bool in = s < a.n_parts && in_bounds(a.fault, row * a.n_parts + s, n_part_rows(a));
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
  if (!in_bounds(a.fault, row, n_rows(a))) return;
  const float4 y = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x / L, acc.y / L, acc.z / L, acc.w / L);
  store_four(a.out, a.out_dtype, row * kHeadDim + 4 * lane, y);
  if (lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int RB, bool kWide>
cudaError_t run(const ServeArgs& a, dim3 grid, cudaStream_t stream) {
  static PerDeviceFlag flag;
  const size_t bytes = (static_cast<size_t>(RB) * kPad + kTile * kPad + kTile * kHeadDim) * sizeof(float);
  static_assert(RB <= kPad, "the weights fit over the keys");
  const cudaError_t e = set_smem_limit_once(flag, attend_f32_kernel<RB, kWide>, bytes);
  if (e != cudaSuccess) return e;
  return launch_chained(attend_f32_kernel<RB, kWide>, grid, kThreads, a, stream, bytes);
}

}  // namespace

cudaError_t launch_prefix_f32(const ServeArgs& a, cudaStream_t stream) {
  const int rows = a.batch * a.group;
  const dim3 grid(a.n_splits, a.n_kv_heads, rows <= 16 ? 1 : (rows + 63) / 64);
  if (rows <= 16) return a.wide ? run<16, true>(a, grid, stream) : run<16, false>(a, grid, stream);
  return a.wide ? run<64, true>(a, grid, stream) : run<64, false>(a, grid, stream);
}

cudaError_t launch_merge(const ServeArgs& a, cudaStream_t stream) {
  return launch_chained(merge_kernel, dim3(static_cast<unsigned>(a.batch) * a.n_q_heads), 32 * kMergeWarps, a, stream);
}

}  // namespace cvq
