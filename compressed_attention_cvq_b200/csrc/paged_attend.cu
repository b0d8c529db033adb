// cvq_paged_attend: decode attention over 16-bit pages, one launch.
//
// What bounds it: every cached key and value is read once and used by the g = Hq/Hkv query
// heads of its KV head, 4 g FMA per 4 bytes, so device memory is the floor as long as the
// arithmetic stays out of the way.  On the CUDA cores it does not (g = 8 would take two
// thirds of the FP32 rate), so the products run as 16-bit matrix instructions of 16 x 8 x 16
// (mma.sync: the 16 rows of a decode step fill no 128-row tcgen05 tile, and at this shape a
// tenth of the issue slots suffices).
//
// Exactness: rows 0-7 of the 16-row operand hold the g heads, rows 8-15 the same heads'
// remainders -- a query or weight x is split as hi = 16-bit(x), lo = 16-bit(x - hi), and the two
// result rows are added.  So fp32 queries, queries of the other 16-bit type and the softmax
// weights keep 16 bits (bf16 pages) or 22 bits (fp16 pages) at no extra instruction, since a
// group has at most 8 heads.  Where queries or outputs are fp32 and a group has at most 4 heads
// (kFine), the rows that are left, 4-7, take a third part (24 bits), and a warp adds its outputs to
// an fp32 copy in shared memory every 64 chunks, since the accumulators of the matrix instructions
// do not round to nearest: over 16384 tokens outputs are off by 1.0e-6 instead of 4.0e-6 (fp32
// arithmetic 1.7e-6) at 494 us instead of 485.
// For fp16 pages a query row is first scaled by a power of two into fp16's range, and the weights
// are taken relative to 2^15 below the maximum, so that the small ones stay normal numbers.  bf16
// has fp32's range: there they are taken relative to 2^-8, so that sums of the largest values have
// room.  Scores, weights' sums and outputs accumulate in fp32.
//
// Measured in a captured graph, 8 KV heads, bf16 pages: 64 sequences of up to 16384 tokens 494 us
// (6.5 TB/s, the rate of a copy; fp32 queries), one of 131071 (fp16) 89 us (6.0 TB/s), 16 of 1024 to 8192 54 us
// (5.7 TB/s), 32 of up to 128 7.2 us.
//
// Split: a CTA of 4 warps takes one (sequence, KV head, run of tokens); a warp
// takes every fourth chunk of 16 tokens through its own ring of cp.async stages (keys and
// values of a chunk, 8 KB), so that no CTA barrier runs in the loop, and keeps its own
// maximum, sum and output; the four are joined through shared memory at the end.  A CTA whose
// split starts behind its sequence leaves at once, and the CTA of a (sequence, KV head) that
// finishes last merges the splits (as in cvq_attend; the order of the sum is fixed).
#include <type_traits>

#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMinSplit = 256;                    // tokens that are worth a CTA and its part of a merge
constexpr int kChunk = 16;                        // tokens of a stage
constexpr int kStages = 3;                        // two in flight; 2, 4 and 5 measured slower
constexpr int kRowBytes = 2 * kHeadDim;
constexpr int kTileBytes = kChunk * kRowBytes;    // keys or values of a stage
constexpr int kRingBytes = kStages * 2 * kTileBytes;
constexpr int kSmemBytes = kWarps * kRingBytes;
constexpr int kRun = 64;                          // chunks between flushes of a warp's outputs (kFine)
constexpr int kCtasPerSm = 2;                     // 96 KB of ring each
static_assert(kRingBytes >= 8 * kHeadDim * 4, "a warp's output fits its ring");

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool have) {
  const int bytes = have ? 16 : 0;                // 0: nothing is read, 16 zero bytes land
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x and y as a pair of 16-bit numbers; x and y become their remainders
template <typename T>
__device__ __forceinline__ uint32_t take_part(float& x, float& y);
template <>
__device__ __forceinline__ uint32_t take_part<__nv_bfloat16>(float& x, float& y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  x -= __low2float(h);
  y -= __high2float(h);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t take_part<__half>(float& x, float& y) {
  const __half2 h = __floats2half2_rn(x, y);
  x -= __low2float(h);
  y -= __high2float(h);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// out and lse of one row from its sum (M in log2 units, L, and lane's 4 dims of o), with the
// earlier state of the row if there is one
__device__ __forceinline__ void finish_row(const ServeArgs& a, size_t row, int lane, float M, float L, float4 o) {
  if (!in_bounds(a.fault, row, n_rows(a))) return;
  if (a.prev_lse != nullptr) {
    const float pz = a.prev_lse[row] * kLog2e;
    if (pz != -INFINITY) {
      const float4 po = *reinterpret_cast<const float4*>(a.prev_out + row * kHeadDim + 4 * lane);
      const float mn = fmaxf(M, pz);
      const float f = M == -INFINITY && L == 0.f ? 0.f : exp2f(M - mn), p = exp2f(pz - mn);
      o = make_float4(o.x * f + po.x * p, o.y * f + po.y * p, o.z * f + po.z * p, o.w * f + po.w * p);
      L = L * f + p;
      M = mn;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t at = row * kHeadDim + 4 * lane;
  const float x[4] = {L == 0.f ? 0.f : o.x * inv, L == 0.f ? 0.f : o.y * inv,
                      L == 0.f ? 0.f : o.z * inv, L == 0.f ? 0.f : o.w * inv};
  __syncwarp();                                   // prev_lse may be lse
  store_four(a.out, a.out_dtype, at, make_float4(x[0], x[1], x[2], x[3]));
  if (lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <typename T, bool kFine>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_attend_kernel(const __grid_constant__ ServeArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t s_mask[kWarps][kStages];
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  __shared__ int s_last, s_longest[kWarps];
  static_assert(kWarps == 4, "the maximum below");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid = lane & 3;      // fragment row and column pair
  const int head = kFine ? gid & 3 : gid;         // of the group
  const bool upper = kFine && gid >= 4;           // rows with the third parts
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int L = a.lens[b];
  L = L < 0 ? 0 : (L > a.t_cap ? a.t_cap : L);
  // Splits are shares of the longest sequence, whatever the page table has room for: shorter ones
  // take fewer splits, so that CTAs carry like amounts (16 sequences of 1024 to 8192: 53 us; every
  // sequence in equal parts: 58 us).
  int longest = L;
  if (a.n_splits > 1) {
    int x = 0;
    for (int i = threadIdx.x; i < a.batch; i += kThreads) x = max(x, __ldg(a.lens + i));
    x = __reduce_max_sync(0xffffffffu, x);
    if (lane == 0) s_longest[warp] = x;
    __syncthreads();
    longest = min(max(max(s_longest[0], s_longest[1]), max(s_longest[2], s_longest[3])), a.t_cap);
  }
  const long long share = (static_cast<long long>(longest) + a.n_splits - 1) / a.n_splits;
  const long long per64 = max(static_cast<long long>(kMinSplit), (share + kSplitAlign - 1) / kSplitAlign * kSplitAlign);
  const int per = static_cast<int>(min(per64, 0x7fffffffLL));               // one split holds any length
  const int used = L == 0 ? 1 : static_cast<int>((static_cast<long long>(L) + per - 1) / per);     // splits that hold tokens
  if (split >= used) return;
  const int start = split * per;                  // < L
  const int end = min(L - start, per) + start;
  const int nchunks = (end - start + kChunk - 1) / kChunk;
  const size_t row0 = static_cast<size_t>(b) * a.n_q_heads + static_cast<size_t>(h) * a.group;

  // ---- copies ----
  const int* table = a.page_table + static_cast<size_t>(b) * a.max_pages;
  const uint32_t ring = smem_u32(smem) + warp * kRingBytes;
  const int slot_mask = (1 << a.page_shift) - 1;
  // token lane & 15 of chunk i (a chunk may pass 2^31 where the sequence ends just before), and its
  // page, loaded one chunk ahead of its use
  auto token = [&](int i) { return static_cast<unsigned>(start) + static_cast<unsigned>(i) * kChunk + (lane & 15); };
  auto load_page = [&](int i) {
    const unsigned t = token(i);
    return i < nchunks && t < static_cast<unsigned>(end) && in_bounds(a.fault, t >> a.page_shift, a.max_pages)
               ? __ldg(table + (t >> a.page_shift)) : 0;
  };
  auto issue = [&](int i, int page) {
    if (i < nchunks) {
      const unsigned t = token(i);
      const bool in_range = static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
      const bool mine = t < static_cast<unsigned>(end), have = mine && in_range;
      if (mine && !in_range) atomicOr(a.fault, kFaultPage);
      const uint32_t mask = __ballot_sync(0xffffffffu, have) & 0xffffu;
      const long long off = have ? static_cast<long long>(page) * a.page_stride +
                                       (static_cast<long long>(h) * (slot_mask + 1) + (t & slot_mask)) * kHeadDim
                                 : 0;
      const uint32_t stage = ring + (i / kWarps % kStages) * (2 * kTileBytes);
      if (lane == 0) s_mask[warp][i / kWarps % kStages] = mask;
      const int half = lane >> 4, col = lane & 15;
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        const int r = 2 * j + half;
        const long long o = __shfl_sync(0xffffffffu, off, r) + 8 * col;
        const bool ok = (mask >> r) & 1u;
        const uint32_t dst = stage + r * kRowBytes + ((col ^ (r & 7)) << 4);
        cp16(dst, static_cast<const uint16_t*>(a.k_pages) + o, ok);
        cp16(dst + kTileBytes, static_cast<const uint16_t*>(a.v_pages) + o, ok);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int page = load_page(warp);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    const int i = warp + s * kWarps;
    const int next = load_page(i + kWarps);
    issue(i, page);
    page = next;
  }

  // the parts of x and y that belong in this lane's rows: gid, and gid + 8
  auto parts = [&](float x, float y, uint32_t& low_row, uint32_t& high_row) {
    low_row = take_part<T>(x, y);
    high_row = take_part<T>(x, y);
    if constexpr (kFine) {
      const uint32_t third = take_part<T>(x, y);
      if (upper) {
        low_row = third;
        high_row = 0u;
      }
    }
  };

  // ---- the query operand ----
  uint32_t qa[8][4];
  float factor = 0.08838834764831845f * kLog2e;   // of a product of the operand rows
  {
    float x[8][4];
    const size_t at = (row0 + head) * kHeadDim;
    float mx = 0.f;
#pragma unroll
    for (int kt = 0; kt < 8; ++kt) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = kt * 16 + 2 * tid + (j & 1) + (j >> 1) * 8;
        x[kt][j] = head < a.group && in_bounds(a.fault, row0 + head, n_rows(a)) ? load_any(a.q, a.q_dtype, at + d) : 0.f;
        mx = fmaxf(mx, fabsf(x[kt][j]));
      }
    }
    float down = 1.f;
    if (sizeof(T) == 2 && a.kv_dtype == CVQ_F16) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (mx > 0.f && mx < INFINITY) {
        // 2^-e for mx in [2^e, 2^(e+1)); e is kept to where both powers are normal numbers
        const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -120), 120);
        down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        factor *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      }
    }
#pragma unroll
    for (int kt = 0; kt < 8; ++kt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float u = x[kt][2 * j] * down, v = x[kt][2 * j + 1] * down;
        parts(u, v, qa[kt][2 * j], qa[kt][2 * j + 1]);
      }
    }
  }

  // ---- one pass over this warp's chunks ----
  // weights are 2^(s - ref), ref = running maximum - kLift
  constexpr float kLift = std::is_same<T, __half>::value ? 15.f : -8.f;
  float m = -INFINITY, l = 0.f;
  float o[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[n][j] = 0.f;
  // kFine: this lane's outputs so far, added in fp32 and taken to the maximum of now
  float* kept = reinterpret_cast<float*>(smem + kSmemBytes) + warp * (4 * kHeadDim);
  float m_kept = -INFINITY;
  int run = 0;
  bool any = false;
  auto flush = [&] {
    const float f = m_kept == -INFINITY ? 0.f : exp2f(m_kept - m);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      float u = o[n][0] + o[n][2], v = o[n][1] + o[n][3];
      u += __shfl_xor_sync(0xffffffffu, u, 16);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (!upper) {
        float2* at = reinterpret_cast<float2*>(kept + gid * kHeadDim + 8 * n + 2 * tid);
        const float2 x = any ? *at : make_float2(0.f, 0.f);
        *at = make_float2(fmaf(x.x, f, u), fmaf(x.y, f, v));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][j] = 0.f;
    }
    m_kept = m;
    run = 0;
    any = true;
  };
  for (int i = warp; i < nchunks; i += kWarps) {
    const int ahead = i + (kStages - 1) * kWarps;
    const int next = load_page(ahead + kWarps);
    issue(ahead, page);
    page = next;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t stage = ring + (i / kWarps % kStages) * (2 * kTileBytes);
    const uint32_t mask = s_mask[warp][i / kWarps % kStages];
    float c[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[n][j] = 0.f;
    {
      const int r = (lane & 7) + ((lane >> 4) << 3), sel = (lane >> 3) & 1;
#pragma unroll
      for (int kt = 0; kt < 8; ++kt) {
        uint32_t kb[4];
        ldsm4(kb, stage + r * kRowBytes + (((2 * kt + sel) ^ (r & 7)) << 4));
        mma16<T>(c[0], qa[kt], kb[0], kb[1]);
        mma16<T>(c[1], qa[kt], kb[2], kb[3]);
      }
    }
    float s[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[n][j] = c[n][j] + c[n][j + 2];
        if (kFine) s[n][j] += __shfl_xor_sync(0xffffffffu, s[n][j], 16);
        s[n][j] *= factor;
        if (mask != 0xffffu && !((mask >> (8 * n + 2 * tid + j)) & 1u)) s[n][j] = -INFINITY;
      }
    float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx > m)) {
      const float mn = fmaxf(m, mx);
      const float alpha = mn == -INFINITY ? 1.f : exp2f(m - mn);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][j] *= alpha;
    }
    const float ref = m == -INFINITY ? 0.f : m - kLift;
    float p[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[n][j] = exp2f(s[n][j] - ref);
        l += p[n][j];
      }
    uint32_t pa[4];
    parts(p[0][0], p[0][1], pa[0], pa[1]);
    parts(p[1][0], p[1][1], pa[2], pa[3]);
    {
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), sel = lane >> 4;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        uint32_t vb[4];
        ldsm4t(vb, stage + kTileBytes + r * kRowBytes + (((2 * n + sel) ^ (r & 7)) << 4));
        mma16<T>(o[2 * n], pa, vb[0], vb[1]);
        mma16<T>(o[2 * n + 1], pa, vb[2], vb[3]);
      }
    }
    __syncwarp();                                 // the stage may be refilled
    if constexpr (kFine) {
      if (++run == kRun) flush();
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  __syncwarp();

  // ---- join the warps: each leaves [8 heads][128] and its maximum and sum ----
  if constexpr (kFine) {
    flush();
  } else {
    float* mine = reinterpret_cast<float*>(smem + warp * kRingBytes);
#pragma unroll
    for (int n = 0; n < 16; ++n)
      *reinterpret_cast<float2*>(mine + gid * kHeadDim + 8 * n + 2 * tid) =
          make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
  }
  auto left_by = [&](int w) {
    return reinterpret_cast<const float*>(kFine ? smem + kSmemBytes + w * (4 * kHeadDim * 4) : smem + w * kRingBytes);
  };
  if (tid == 0) {
    s_m[warp][gid] = m == -INFINITY ? -INFINITY : m - kLift;
    s_l[warp][gid] = l;
  }
  __syncthreads();
  for (int r = warp; r < a.group; r += kWarps) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (s_m[w][r] == -INFINITY && s_l[w][r] == 0.f) continue;             // no token
      const float f = exp2f(s_m[w][r] - M);
      const float4 x = *reinterpret_cast<const float4*>(left_by(w) + r * kHeadDim + 4 * lane);
      sum = fmaf(s_l[w][r], f, sum);
      acc = make_float4(fmaf(x.x, f, acc.x), fmaf(x.y, f, acc.y), fmaf(x.z, f, acc.z), fmaf(x.w, f, acc.w));
    }
    if (used == 1) {
      finish_row(a, row0 + r, lane, M, sum, acc);
    } else {
      const size_t at = (row0 + r) * a.n_splits + split;
      if (!in_bounds(a.fault, at, n_part_rows(a))) continue;
      *reinterpret_cast<float4*>(a.part_o + at * kHeadDim + 4 * lane) = acc;
      if (lane == 0) {
        a.part_m[at] = M;
        a.part_l[at] = sum;
      }
    }
  }
  if (used == 1) return;

  // ---- the last CTA of this (sequence, KV head) merges its splits ----
  __syncthreads();
  const size_t unit = static_cast<size_t>(b) * a.n_kv_heads + h;
  if (!in_bounds(a.fault, unit, kCounters)) return;         // the same for all threads
  int* counter = a.counters + unit;
  if (threadIdx.x == 0) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    s_last = old == used - 1;
  }
  __syncthreads();
  if (!s_last) return;
  // W = 4 / g warps share a row (g <= 4; at g = 8 a warp takes two rows), 4 dims a lane; one
  // pass over the splits, U of them in flight
  float4* part = reinterpret_cast<float4*>(smem);                           // [warps][32]
  const int W = a.group >= kWarps ? 1 : kWarps / a.group;
  for (int r = warp / W; r < a.group; r += kWarps / W) {
    const float* pm = a.part_m + (row0 + r) * a.n_splits;
    const float* pl = a.part_l + (row0 + r) * a.n_splits;
    const float4* po = reinterpret_cast<const float4*>(a.part_o + (row0 + r) * a.n_splits * kHeadDim) + lane;
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;
    for (int s0 = warp % W; s0 < used; s0 += U * W) {
      float4 x[U];
      float mv[U], lv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * W;
        const bool in = s < used && in_bounds(a.fault, (row0 + r) * a.n_splits + s, n_part_rows(a));
        mv[u] = in ? __ldcg(pm + s) : -INFINITY;
        lv[u] = in ? __ldcg(pl + s) : 0.f;
        x[u] = in ? __ldcg(po + static_cast<size_t>(s) * (kHeadDim / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mn = M;
#pragma unroll
      for (int u = 0; u < U; ++u) mn = fmaxf(mn, mv[u]);
      const float alpha = mn == -INFINITY ? 1.f : exp2f(M - mn);
      M = mn;
      sum *= alpha;
      acc = make_float4(acc.x * alpha, acc.y * alpha, acc.z * alpha, acc.w * alpha);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = mv[u] == -INFINITY && lv[u] == 0.f ? 0.f : exp2f(mv[u] - M);
        sum = fmaf(lv[u], f, sum);
        acc = make_float4(fmaf(x[u].x, f, acc.x), fmaf(x[u].y, f, acc.y), fmaf(x[u].z, f, acc.z), fmaf(x[u].w, f, acc.w));
      }
    }
    if (W == 1) {
      finish_row(a, row0 + r, lane, M, sum, acc);
    } else {
      part[warp * 32 + lane] = acc;
      if (lane == 0) {
        s_m[warp][0] = M;
        s_l[warp][0] = sum;
      }
    }
  }
  if (W > 1) {
    __syncthreads();
    const int r = warp;                                                     // g = 1 or 2 rows
    if (r < a.group) {
      float M = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = r * W; w < (r + 1) * W; ++w) M = fmaxf(M, s_m[w][0]);
      for (int w = r * W; w < (r + 1) * W; ++w) {
        if (s_m[w][0] == -INFINITY && s_l[w][0] == 0.f) continue;
        const float f = exp2f(s_m[w][0] - M);
        const float4 x = part[w * 32 + lane];
        sum = fmaf(s_l[w][0], f, sum);
        acc = make_float4(fmaf(x.x, f, acc.x), fmaf(x.y, f, acc.y), fmaf(x.z, f, acc.z), fmaf(x.w, f, acc.w));
      }
      finish_row(a, row0 + r, lane, M, sum, acc);
    }
  }
  if (threadIdx.x == 0) atomicExch(counter, 0);
}

template <typename T, bool kFine>
cudaError_t run(const ServeArgs& a, cudaStream_t stream) {
  static PerDeviceFlag flag;
  constexpr size_t bytes = kSmemBytes + (kFine ? kWarps * 4 * kHeadDim * sizeof(float) : 0);
  const cudaError_t e = set_smem_limit_once(flag, paged_attend_kernel<T, kFine>, bytes);
  if (e != cudaSuccess) return e;
  return launch_chained(paged_attend_kernel<T, kFine>, dim3(a.n_splits, a.n_kv_heads, a.batch), kThreads, a, stream, bytes);
}

}  // namespace

cudaError_t launch_paged_attend(const ServeArgs& a, cudaStream_t stream) {
  const bool fine = a.group <= 4 && (a.q_dtype == CVQ_F32 || a.out_dtype == CVQ_F32);
  if (a.kv_dtype == CVQ_BF16) return fine ? run<__nv_bfloat16, true>(a, stream) : run<__nv_bfloat16, false>(a, stream);
  return fine ? run<__half, true>(a, stream) : run<__half, false>(a, stream);
}

}  // namespace cvq
