// Shared-prefix attention of 16-bit queries on the tensor cores: each cached token is decoded
// from its codes once per KV head, as fp16, straight into the operand tiles of the matrix
// products, and read there by the query rows of every sequence.
//
// A CTA takes 128 query rows ((sequence, head of the group) pairs) of a KV head and a run of
// tokens, in tiles of 64:
//   producers (8 warps for keys, 4 or 8 for values)  gather codewords from fp16 codebooks in
//                        shared memory, sum the rounds, rotate the keys and store the tiles
//   one thread           copies codes, steps ahead, into shared memory (8-scalar groups)
//   two threads          S = Q K^T (M = 128 rows, N = 64 tokens; Q from TMEM), O += P V
//                        (N = 128 dims; P from TMEM), both tcgen05.mma kind::f16
//   softmax (2 x 4 warps)  a thread owns a row: even tiles go to the first four warps, odd
//                        ones to the others, each with its own O, maximum and sum (joined at
//                        the end), so that the exponentials of one tile run under the other's
//                        loads and barriers
// What bounds it: for 128 rows no one unit (the exponentials, the products, the FMA pipe and the
// gathers take a fifth to a third of their rates each, the issue slots half); for fewer rows the
// producers.  Measured in a captured graph, 32 query and 8 KV heads: 32 sequences over 131072
// tokens, R = 1, 105 us (660 TFLOP/s of 1646, the floor is 42 us); 16 over 32768, R = 2, 43 us, and
// R = 11 of 64-scalar groups 111 us; a short prefix 12 us, of which the first tile's scores come
// after 5 (the codebooks' conversion 3) and the join and merge take 4.
//
// Bank conflicts: codebooks lie as [round][code][chunk of 8 dims], so 8 lanes that work on the
// 8 (or 16) chunks of one token read 8 different bank groups whatever their codes are.
//
// Codebooks that exceed one SM (two rounds of 8-scalar groups, 64-scalar groups) are split by
// dims over a pair of CTAs: each decodes its 64 dims of both CTAs' tokens and stores the other
// CTA's half through distributed shared memory (st.async: 53 us where stores and a fence took 97).
// Of more than 11 rounds of 64-scalar groups the others are gathered from the workspace's copy of
// the codebooks, from L2 (16 sequences over 4096 tokens, R = 21: 56 us; in fp32 151).
//
// Phases: a producer thread keeps e^{i theta t} of its 4 pairs in fp32 and turns them on from
// token to token; every 64 tiles they are taken anew from the exact turns, which holds their
// error below 2^-15 (2^-19 typical), far under the operands' 2^-12.
//
// Roundings to fp16, 2^-11 at most each: a codeword; the sum of two codewords of 8-scalar groups
// and of neighbouring rounds of 64-scalar groups (the rounds' total is fp32 there); for 8-scalar
// groups the sine and cosine and the two products of a rotation, whose fp16 arithmetic takes half
// the instructions of fp32 and conversions (124 us -> 116); the rotated key; the value; the
// weight.  A score is then off by 5e-4 of its terms' root mean square, a value by 3e-4, at random
// from token to token: below bf16's own rounding of the output, and averaged over the softmax in
// lse.  Codebooks and query rows are scaled by powers of two into fp16's range.  Products are
// summed, and the softmax, O and the merge kept, in fp32.
#include <type_traits>

#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kSoftWarps = 8;
// The warps by their roles.
template <bool kWide>
struct Roles {
  static constexpr int kKeyWarps = 8, kValueWarps = kWide ? 8 : 4;
  static constexpr int kValueWarp = kSoftWarps + kKeyWarps;                   // the first
  static constexpr int kScoreWarp = kValueWarp + kValueWarps, kOutWarp = kScoreWarp + 1, kCopyWarp = kOutWarp + 1;
  static constexpr int kThreads = 32 * (kCopyWarp + 1);
};
constexpr int kRows = 128;
constexpr int kTok = 64;                          // tokens of a tile
constexpr int kHalfTile = kTok * 128;             // 64 dims of its keys or values, bytes
constexpr int kTile = 2 * kHalfTile;
constexpr int kMostCodeStages = 8;                // what a CTA alone has room for; a pair has for 4
constexpr int kReanchor = 64;                     // tiles between exact phases
constexpr int kOutPitch = kHeadDim + 4;           // floats; 16-byte chunks of 8 rows in 8 bank groups
constexpr int kOutBytes = kRows * kOutPitch * 4;
// columns of TMEM: S of the two streams, their P (two fp16 a column), Q, their O
constexpr uint32_t kColS = 0, kColP = 128, kColQ = 192, kColO = 256, kTmemCols = 512;

struct Control {
  uint64_t book;                                  // codebooks
  uint64_t q_full;
  uint64_t c_full[2][kMostCodeStages], c_empty[2][kMostCodeStages];         // codes of keys, values
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full[2], pv_done[2];
  uint32_t tmem;
  alignas(16) float turn[16][8];                  // steps (and jumps) of the phases, per chunk
  float m[2][kRows], l[2][kRows];                 // the streams' states
};

// ---- PTX ----
__device__ __forceinline__ bool try_wait(uint32_t bar, unsigned parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}
// the bounded rest of a wait, out of line: the waits are in every role's loop
__device__ __noinline__ bool wait_on(uint32_t bar, unsigned parity, unsigned int* fault) {
  unsigned long long t0 = 0;
  for (unsigned i = 1;; ++i) {
    if (try_wait(bar, parity)) return true;
    if (i % 64 == 0) {                            // the clock is slow to read: now and then
      unsigned long long now;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      if (t0 == 0) t0 = now;
      else if (now - t0 > kMbarWaitLimitNs) {
        atomicOr(fault, kFaultCopyTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(uint64_t* bar, unsigned parity, unsigned int* fault) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (try_wait(addr, parity)) return true;
  return wait_on(addr, parity, fault);
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int C>
__device__ __forceinline__ void commit(uint64_t* bar, bool both) {
  if (C == 2 && both) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3)) : "memory");
  } else {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
  }
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(static_cast<uint32_t>(acc)) : "memory");
}
#define CVQ_R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define CVQ_V4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : CVQ_R4(r, 0), CVQ_R4(r, 4), CVQ_R4(r, 8), CVQ_R4(r, 12), CVQ_R4(r, 16), CVQ_R4(r, 20), CVQ_R4(r, 24), CVQ_R4(r, 28)
      : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : CVQ_R4(r, 0), CVQ_R4(r, 4), CVQ_R4(r, 8), CVQ_R4(r, 12) : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::CVQ_V4(r, 0),
               CVQ_V4(r, 4), CVQ_V4(r, 8), CVQ_V4(r, 12), "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::CVQ_V4(r, 0), CVQ_V4(r, 4), "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// operand descriptor: 128-byte swizzle, `lead` and `stride` bytes (see the tiles' layouts below)
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// to the other CTA; its barrier counts the bytes as they land, so that nothing waits for them here
__device__ __forceinline__ void send16(uint32_t addr, uint4 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(addr), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes != 0;
}
// pairs of fp32 numbers in one instruction
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1,%2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack(f2 v) {
  float2 r;
  asm("mov.b64 {%0,%1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 x, f2 y) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 x, f2 y, f2 z) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ f2 add2(f2 x, f2 y) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ f2 neg2(f2 x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for -126 <= e <= 127, and floor(log2 x) of a normal number
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ int log2_floor(float x) { return static_cast<int>(__float_as_uint(x) >> 23 & 255) - 127; }
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 floats_of(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
__device__ __forceinline__ uint32_t add_halves(uint32_t x, uint32_t y) {
  const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x[8] += the 8 fp16 numbers of v
__device__ __forceinline__ void add_chunk(float (&x)[8], uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("add.f32.f16 %0, %1, %0;" : "+f"(x[2 * i]) : "h"(static_cast<uint16_t>(w[i] & 0xffffu)));
    asm("add.f32.f16 %0, %1, %0;" : "+f"(x[2 * i + 1]) : "h"(static_cast<uint16_t>(w[i] >> 16)));
  }
}
__device__ __forceinline__ uint4 add_chunks(uint4 x, uint4 y) {
  return make_uint4(add_halves(x.x, y.x), add_halves(x.y, y.y), add_halves(x.z, y.z), add_halves(x.w, y.w));
}

// e^{i theta_j t} of the 4 pairs of a chunk; packed two pairs at a time
struct Phase {
  f2 c[2], s[2];
  __device__ __forceinline__ void set(const PhaseTurns& ph, int chunk, unsigned long long t) {
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = phase_exact(ph.F[4 * chunk + j] * t);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      c[p] = pack(v[2 * p].x, v[2 * p + 1].x);
      s[p] = pack(v[2 * p].y, v[2 * p + 1].y);
    }
  }
  // 8 floats in shared memory: the 4 cosines, then the 4 sines
  __device__ __forceinline__ void put(uint32_t at) const {
    const float2 c0 = unpack(c[0]), c1 = unpack(c[1]), s0 = unpack(s[0]), s1 = unpack(s[1]);
    sts16(at, make_uint4(__float_as_uint(c0.x), __float_as_uint(c0.y), __float_as_uint(c1.x), __float_as_uint(c1.y)));
    sts16(at + 16, make_uint4(__float_as_uint(s0.x), __float_as_uint(s0.y), __float_as_uint(s1.x), __float_as_uint(s1.y)));
  }
  __device__ __forceinline__ void get(uint32_t at) {
    const uint4 x = lds16(at), y = lds16(at + 16);
    c[0] = pack(__uint_as_float(x.x), __uint_as_float(x.y));
    c[1] = pack(__uint_as_float(x.z), __uint_as_float(x.w));
    s[0] = pack(__uint_as_float(y.x), __uint_as_float(y.y));
    s[1] = pack(__uint_as_float(y.z), __uint_as_float(y.w));
  }
  __device__ __forceinline__ void turn(const Phase& w) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const f2 nc = fma2(neg2(s[p]), w.s[p], mul2(c[p], w.c[p]));
      s[p] = fma2(s[p], w.c[p], mul2(c[p], w.s[p]));
      c[p] = nc;
    }
  }
  // 8 dims of a key, in the order re re im im re re im im, rotated and rounded
  __device__ __forceinline__ uint4 rotate(const float (&x)[8]) const {
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const f2 re = pack(x[4 * p], x[4 * p + 1]), im = pack(x[4 * p + 2], x[4 * p + 3]);
      const float2 a = unpack(fma2(im, neg2(s[p]), mul2(re, c[p]))), b = unpack(fma2(im, c[p], mul2(re, s[p])));
      w[2 * p] = half_pair(a.x, a.y);
      w[2 * p + 1] = half_pair(b.x, b.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // the same in fp16 arithmetic
  __device__ __forceinline__ uint4 rotate(uint4 k) const {
    const uint32_t in[4] = {k.x, k.y, k.z, k.w};
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float2 cc = unpack(c[p]), ss = unpack(s[p]);
      const __half2 co = __floats2half2_rn(cc.x, cc.y), si = __floats2half2_rn(ss.x, ss.y);
      const __half2 re = *reinterpret_cast<const __half2*>(&in[2 * p]), im = *reinterpret_cast<const __half2*>(&in[2 * p + 1]);
      const __half2 a = __hfma2(__hneg2(im), si, __hmul2(re, co)), b = __hfma2(im, co, __hmul2(re, si));
      w[2 * p] = *reinterpret_cast<const uint32_t*>(&a);
      w[2 * p + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// ---- codebooks ----
// A CTA holds chunk (of 8 dims) * entry items of 16 bytes: i -> [round][entry][chunk] of its CH
// chunks, which for a 64-scalar group is the codebook's own order.
template <int C, bool kWide>
__device__ __forceinline__ const float* book_item(const float* cb, int R, int rank, int i) {
  constexpr int CH = 16 / C;
  if (kWide) return cb + (static_cast<size_t>(rank) * R * kWideCodes * 8 + i) * 8;
  const int chunk = i % CH + (C == 2 ? 8 * rank : 0);
  return cb + (static_cast<size_t>(chunk) * R * kCodes + i / CH) * 8;
}
template <int C, bool kWide>
__host__ __device__ constexpr int book_items(int R) {
  return kWide ? R * kWideCodes * 8 : R * kCodes * (16 / C);
}
// Keys are held, here and in the operand tiles, with the two real and the two imaginary parts of
// two pairs side by side, so that a pair of fp16 numbers rotates in one instruction each.
template <bool kWide>
__host__ __device__ constexpr int held_rounds(int R) {
  return kWide && R > kWideRoundsPerCta ? kWideRoundsPerCta : R;
}
__device__ __forceinline__ uint4 scaled_halves(float4 x, float4 y, float scale, bool keys) {
  if (keys) {
    const float4 a = x, b = y;
    x = make_float4(a.x, a.z, a.y, a.w);
    y = make_float4(b.x, b.z, b.y, b.w);
  }
  return make_uint4(half_pair(x.x * scale, x.y * scale), half_pair(x.z * scale, x.w * scale),
                    half_pair(y.x * scale, y.y * scale), half_pair(y.z * scale, y.w * scale));
}

// Exponent of the codebook scale: 6 wherever the decoded numbers then lie well inside fp16's
// range, so that one reading of the codebook is enough; else what takes the largest to 2^14.
constexpr int kUsualScale = 6;
constexpr int kBookThreads = 256;

// The codebooks as CTAs of the attention kernel hold them, in fp16 times 2^kUsualScale, into
// the workspace, and the largest finite |x| of every 256 items: converted once a call, and read
// from there by all the CTAs of a KV head in half the bytes.  Launched before the attention
// kernel, whose own set-up runs under it.
template <int C, bool kWide>
__global__ void __launch_bounds__(kBookThreads) prefix_book_kernel(const __grid_constant__ ServeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");                        // for what ran before this call
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t warp_peak[kBookThreads / 32];
  const int n = book_items<C, kWide>(a.R), i = blockIdx.x * kBookThreads + threadIdx.x;
  const int rank = blockIdx.y >> 1, values = blockIdx.y & 1, h = blockIdx.z;
  const float* cb = values ? a.val_cb + static_cast<long long>(h) * a.val_cb_stride
                           : a.key_cb + static_cast<long long>(h) * a.key_cb_stride;
  const float* src = book_item<C, kWide>(cb, a.R, rank, i);
  const float4 x = __ldg(reinterpret_cast<const float4*>(src)), y = __ldg(reinterpret_cast<const float4*>(src) + 1);
  const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t peak = 0;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const uint32_t bits = __float_as_uint(v[d]) & 0x7fffffffu;
    if (bits < 0x7f800000u) peak = max(peak, bits);
  }
  reinterpret_cast<uint4*>(a.book)[((static_cast<size_t>(h) * C + rank) * 2 + values) * n + i] =
      scaled_halves(x, y, static_cast<float>(1 << kUsualScale), !values);
  peak = __reduce_max_sync(0xffffffffu, peak);
  if ((threadIdx.x & 31) == 0) warp_peak[threadIdx.x >> 5] = peak;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kBookThreads / 32; ++w) peak = max(peak, warp_peak[w]);
    a.book_peak[((static_cast<size_t>(h) * 2 + values) * C + rank) * gridDim.x + blockIdx.x] = peak;
  }
}
__device__ __forceinline__ int scale_exponent(uint32_t peak_bits, int R) {
  const float most = __uint_as_float(peak_bits) * static_cast<float>(R) * 1.5f;      // 1.5 > sqrt 2: rotated
  if (peak_bits == 0 || (most < 512.f && most > 0.0078125f)) return kUsualScale;
  return min(max(14 - log2_floor(most), -114), 120);
}

// two 16-bit query elements as floats
__device__ __forceinline__ float2 query_pair(uint32_t w, bool bf16) {
  return bf16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : floats_of(w);
}

// kWide: R is the most rounds; the call's own number is a.R
template <int C, bool kWide, int R>
__global__ void __launch_bounds__(Roles<kWide>::kThreads, 1) prefix_mma_kernel(const __grid_constant__ ServeArgs a) {
  using W = Roles<kWide>;
  constexpr int kThreads = W::kThreads, kScoreWarp = W::kScoreWarp, kCopyWarp = W::kCopyWarp;
  constexpr int kGroupTok = C * kTok;             // tokens of a step of the CTA or pair
  constexpr int CH = 16 / C;
  constexpr int kVStages = kWide ? 1 : 2;
  constexpr int kCodeStages = kMostCodeStages / C;
  static_assert(!kWide || C == 2, "a CTA holds one 64-scalar group");
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t tiles_k = smem_u32(smem), tiles_v = tiles_k + 2 * kTile;
  const uint32_t cb_k = tiles_v + kVStages * kTile;
  const int rounds = kWide ? a.R : R;
  // rounds of a codebook in shared memory; more are gathered from the workspace's copy, from L2
  constexpr int kHeldRounds = held_rounds<kWide>(R);
  const int held = min(rounds, kHeldRounds);
  const uint32_t cb_bytes = kWide ? held * kWideCodes * 128 : R * kCodes * CH * 16;
  const uint32_t cb_v = cb_k + cb_bytes;
  // a stage of codes: keys, then values, [token][round][16 groups] as in the cache
  constexpr uint32_t kCodeBytes = kWide ? 0 : kGroupTok * R * kGroups;
  const uint32_t ring = cb_v + cb_bytes;
  const uint32_t ctl_at = max(ring + kCodeStages * 2 * kCodeBytes - tiles_k, static_cast<uint32_t>(kOutBytes));
  Control& ctl = *reinterpret_cast<Control*>(smem + ctl_at);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = C == 2 ? static_cast<int>(blockIdx.x & 1) : 0;
  const int split = blockIdx.x / C, h = blockIdx.y;
  const int r0 = blockIdx.z * kRows;
  const int nrows = min(kRows, a.batch * a.group - r0);
  const int nact = (nrows + 31) / 32;             // softmax warps with rows, of each stream
  const size_t n_parts = static_cast<size_t>(a.n_parts);
  auto global_row = [&](int r) {
    const int rr = r0 + r;
    return static_cast<size_t>(rr / a.group) * a.n_q_heads + static_cast<size_t>(h) * a.group + rr % a.group;
  };
  int L = a.lens[0];
  L = L < 0 ? 0 : (L > a.t_cap ? a.t_cap : L);
  const long long per = ((L + a.n_splits - 1LL) / a.n_splits + kGroupTok - 1) / kGroupTok * kGroupTok;
  const long long start = min(per * split, static_cast<long long>(L)), end = min(start + per, static_cast<long long>(L));
  const int ntiles = static_cast<int>((end - start + kGroupTok - 1) / kGroupTok);
  if (ntiles == 0) {                              // the same for both CTAs of a pair
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x < nrows) {
      const size_t at = global_row(threadIdx.x) * n_parts + blockIdx.x;
      a.part_m[at] = -INFINITY;
      a.part_l[at] = 0.f;
    }
    return;
  }

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");          // the merge

  // ---- set-up ----
  if (warp == kScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == kCopyWarp && lane == 0) {
    mbar_init(&ctl.book, 1);
    mbar_init(&ctl.q_full, 2 * nact);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.k_full[s], W::kKeyWarps);
      mbar_init(&ctl.v_full[s], W::kValueWarps);
      mbar_init(&ctl.k_empty[s], C);
      mbar_init(&ctl.v_empty[s], C);
      mbar_init(&ctl.s_full[s], 1);
      mbar_init(&ctl.s_empty[s], nact);
      mbar_init(&ctl.p_full[s], nact);
      mbar_init(&ctl.pv_done[s], 1);
    }
#pragma unroll
    for (int s = 0; s < kCodeStages; ++s) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        mbar_init(&ctl.c_full[v][s], 1);
        mbar_init(&ctl.c_empty[v][s], v ? W::kValueWarps : W::kKeyWarps);
      }
    }
  }
  __syncwarp();
  tmem_before_sync();
  if (C == 2) cluster_barrier();                  // the other CTA runs, and its barriers are there
  else __syncthreads();
  tmem_after_sync();
  constexpr uint32_t tmem = 0;                    // all columns: the allocation starts at 0
  // scale exponents of the key and value codebooks of this KV head; after the wait for
  // prefix_book_kernel
  auto book_exponents = [&] {
    const int n = C * book_items<C, kWide>(rounds) / kBookThreads;
    const uint32_t* at = a.book_peak + static_cast<size_t>(h) * 2 * n;
    uint32_t k = 0, v = 0;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) {
      k = max(k, __ldcg(at + i));
      v = max(v, __ldcg(at + n + i));
    }
    return make_int2(scale_exponent(__reduce_max_sync(0xffffffffu, k), rounds), scale_exponent(__reduce_max_sync(0xffffffffu, v), rounds));
  };

  float m = -INFINITY, l = 0.f;                   // softmax: log2 maximum and sum of this thread's row
  int ev = 0;                                     // exponent of the values' scale
  if (warp < kSoftWarps) {
    // ================= softmax =================
    const int st = warp >> 2, q4 = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    // weights are 2^(s - m + kLift); m is followed only when it grows by kSlack, so that O is
    // rescaled a few times and not at every tile, and weights stay below 2^(kLift + kSlack)
    constexpr float kLift = 7.f, kSlack = 8.f;
    if (q4 < nact) {
      // the query operand: the largest element of a row brought to [2^8, 2^9); each stream stores
      // half of the dims.  The loops are rolled: code that runs once costs more to fetch than to run
      int eq;
      {
        const int r = q4 * 32 + lane;
        const bool bf16 = a.q_dtype == CVQ_BF16;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + global_row(min(r, nrows - 1)) * kHeadDim);
        float mx = 0.f;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = __ldg(src + 4 * i + k);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = query_pair(w[j], bf16);
              mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
        }
        eq = mx > 0.f && mx < INFINITY ? 8 - log2_floor(mx) : 0;
        const float up = r < nrows ? pow2(min(eq, 127)) : 0.f, rest = pow2(eq - min(eq, 127));
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {             // 16 dims: 8 columns
          const uint4 v[2] = {__ldg(src + 8 * st + 2 * i), __ldg(src + 8 * st + 2 * i + 1)};
          uint32_t x[8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const float2 f0 = query_pair(w[j], bf16), f1 = query_pair(w[j + 1], bf16);
              x[4 * k + j] = half_pair(f0.x * up * rest, f1.x * up * rest);            // in the keys' order
              x[4 * k + j + 1] = half_pair(f0.y * up * rest, f1.y * up * rest);
            }
          }
          tmem_store8(lanes + kColQ + 32 * st + 8 * i, x);
        }
        tmem_store_wait();
        tmem_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&ctl.q_full);
      }
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const int2 e = book_exponents();
      ev = e.y;
      const int by = min(max(-eq - e.x, -252), 252);
      const float factor = 0.08838834764831845f * kLog2e * pow2(by / 2) * pow2(by - by / 2);
      for (int i = st; i < ntiles; i += 2) {
        const unsigned par = (i >> 1) & 1;
        if (!wait(&ctl.s_full[st], par, a.fault)) break;
        tmem_after_sync();
        // 64 scores, held at once where the registers allow it and else read twice
        constexpr int kHeld = kWide ? 1 : 2;
        const long long left = end - (start + static_cast<long long>(i) * kGroupTok + rank * kTok);
        uint32_t s[kHeld][32];
        auto load_scores = [&](int c, uint32_t (&x)[32]) {
          tmem_load32(x, lanes + kColS + st * kTok + 32 * c);
          tmem_load_wait();
          if (left < kTok) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= left) x[j] = 0xff800000u;
          }
        };
        auto scores_read = [&] {                  // the next scores of this stream may come
          tmem_before_sync();
          __syncwarp();
          if (lane == 0) arrive(&ctl.s_empty[st]);
        };
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 1; c >= 0; --c) {
          load_scores(c, s[c % kHeld]);
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            mx4[j / 2 & 3] = fmaxf(mx4[j / 2 & 3], fmaxf(__uint_as_float(s[c % kHeld][j]), __uint_as_float(s[c % kHeld][j + 1])));
        }
        if (kHeld == 2) scores_read();
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        mx *= factor;
        const bool grow = mx > m + kSlack || (m == -INFINITY && mx > m);
        const float alpha = grow ? exp2f(m - mx) : 1.f;
        if (grow) m = mx;
        const float ref = m == -INFINITY ? 0.f : m - kLift;
        const f2 ff = pack(factor, factor), rr = pack(-ref, -ref);
        if (i >= 2) {                             // the last weights of this stream have been used
          if (!wait(&ctl.pv_done[st], par ^ 1, a.fault)) break;
          tmem_after_sync();
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < kHeadDim; c += 16) {
              uint32_t o[16];
              tmem_load16(o, lanes + kColO + st * kHeadDim + c);
              tmem_load_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_store16(lanes + kColO + st * kHeadDim + c, o);
            }
          }
        }
        f2 sum = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (kHeld == 1 && c == 1) {
            load_scores(1, s[0]);
            scores_read();
          }
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t(&x)[32] = s[c % kHeld];
            const float2 y = unpack(fma2(pack(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), ff, rr));
            const float e0 = exp2_fast(y.x), e1 = exp2_fast(y.y);
            sum = add2(sum, pack(e0, e1));
            p[j] = half_pair(e0, e1);
          }
          tmem_store16(lanes + kColP + st * 32 + 16 * c, p);
        }
        const float2 sums = unpack(sum);
        l = fmaf(l, alpha, sums.x + sums.y);
        tmem_store_wait();
        tmem_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&ctl.p_full[st]);
      }
      // the last product of this stream
      const int n = (ntiles - st + 1) / 2;
      if (n > 0) wait(&ctl.pv_done[st], (n - 1) & 1, a.fault);
      tmem_after_sync();
    }
    if (m != -INFINITY) m -= kLift;
  } else if (warp < kScoreWarp) {
    // ================= producers =================
    // Keys and values are made by warps of their own.
    auto produce = [&](auto is_keys) {
      constexpr bool kKeys = decltype(is_keys)::value;
      constexpr int kWarps = kKeys ? W::kKeyWarps : W::kValueWarps, kFirst = kKeys ? kSoftWarps : W::kValueWarp;
      constexpr int kSlots = 32 * kWarps / CH;    // tokens taken at once
      constexpr int kPer = kGroupTok / kSlots;    // tokens of a thread in a step
      constexpr int kStages = kKeys ? 2 : kVStages;
      static_assert(!kWide || kPer == 4, "a word of codes is 4 tokens");
      static_assert(kWide || kSlots % 8 == 0, "the rows of a thread have the same swizzle");
      const int tid = threadIdx.x - 32 * kFirst, cl = tid % CH, slot = tid / CH;
      const int chunk = C == 2 ? 8 * rank + cl : cl;
      uint64_t* full = kKeys ? ctl.k_full : ctl.v_full;
      uint64_t* empty = kKeys ? ctl.k_empty : ctl.v_empty;
      const uint32_t tiles = kKeys ? tiles_k : tiles_v, book = (kKeys ? cb_k : cb_v) + cl * 16;
      const uint8_t* codes = kKeys ? a.key_codes : a.val_codes;
      // Token u of this thread within a step, and its 16 bytes' place in a tile of its CTA: row
      // token % 64 of CTA token / 64.
      auto token = [&](int u) { return kWide ? kPer * slot + u : slot + u * kSlots; };
      const int row = token(0) % kTok;
      const uint32_t at0 = (chunk >> 3) * kHalfTile + row * 128, swizzle = (chunk & 7) ^ (row & 7);
      const uint32_t away = C == 2 ? map_to(tiles_k, static_cast<uint32_t>(rank ^ 1)) - tiles_k : 0;
      auto store = [&](int s, int u, uint4 v) {
        const uint32_t at = tiles + s * kTile + at0 + (kWide ? u * 128 + ((swizzle ^ u) << 4) : (u * kSlots % kTok) * 128 + (swizzle << 4));
        const int to = kWide ? slot / (kTok / kPer) : u * kSlots / kTok;
        if (C == 1 || to == rank) sts16(at, v);
        else send16(at + away, v, smem_u32(full + s) + away);
      };
      // a stage is full when this CTA's warps have stored and the other CTA's half has landed
      auto publish = [&](int s) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (C == 2 && warp == kFirst) mbar_expect_tx(full + s, kHalfTile);
          else arrive(full + s);
        }
      };
      // phases: this thread's own in registers, what they turn by from token to token and from
      // step to step in shared memory, where a chunk's threads share it
      Phase ph;
      const uint32_t steps = smem_u32(&ctl.turn[cl][0]), jumps = steps + 8 * 32;
      auto anchor = [&](int i) {
        ph.set(a.phase, chunk, static_cast<unsigned long long>(start + static_cast<long long>(i) * kGroupTok + token(0)));
      };
      if (kKeys) {
        if (slot == 0 || (kWide && slot == 1)) {
          ph.set(a.phase, chunk, !kWide ? kSlots : slot == 0 ? 1 : kGroupTok - (kPer - 1));
          ph.put(slot == 0 ? steps : jumps);
        }
        anchor(0);
      }
      // 64-scalar groups: a word holds the codes of this slot's 4 tokens for a round; the 8 threads
      // of a slot load two or three rounds each, a step ahead, and pass them around.  Packed codes: the word
      // is 24 bits from byte t / 4 * 3 of a row, in one or two aligned words; every row and step
      // has the same alignment (t_cap and steps are multiples of 64 tokens)
      constexpr int kWords = kWide ? (R + 7) / 8 : 1;
      uint32_t lo[kWords], hi[kWords];
      const unsigned shift = kWide && a.code_bits == 6 ? (3u * slot & 3u) * 8u : 0u;
      auto load_words = [&](int i) {
        const long long t = start + static_cast<long long>(i) * kGroupTok + 4 * slot;
        const size_t row_bytes = a.code_bits == 6 ? static_cast<size_t>(a.t_cap) / 4 * 3 : static_cast<size_t>(a.t_cap);
        const uint8_t* p = codes + ((static_cast<size_t>(h) * kWideGroups + rank) * rounds + cl) * row_bytes +
                           (a.code_bits == 6 ? t / 4 * 3 - (shift >> 3) : t);
#pragma unroll
        for (int k = 0; k < kWords; ++k, p += 8 * row_bytes) {
          lo[k] = hi[k] = 0u;
          if (cl + 8 * k < rounds && t < end) {
            lo[k] = __ldg(reinterpret_cast<const uint32_t*>(p));
            if (shift > 8) hi[k] = __ldg(reinterpret_cast<const uint32_t*>(p) + 1);
          }
        }
      };
      // offset of the codeword of word w and token u within a round of a codebook
      const int unit = a.code_bits == 6 ? 6 : 8;
      auto entry = [&](uint32_t w, int u) { return ((w >> (unit * u)) & 63u) * 128u; };
      // 8-scalar groups: codes from the ring (behind the last token any byte, all of them entries)
      const uint32_t my_codes = ring + (kKeys ? 0 : kCodeBytes) + token(0) * (R * kGroups) + chunk;
      auto code = [&](int i, int u, int r) {
        uint32_t x;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x)
                     : "r"(my_codes + (i % kCodeStages) * (2 * kCodeBytes) + u * (kSlots * R * kGroups) + r * kGroups));
        return x;
      };
      if (kWide) load_words(0);
      if (kKeys) asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const int2 both = book_exponents();
      const int e = kKeys ? both.x : both.y;
      wait(&ctl.book, 0, a.fault);
      if (e != kUsualScale) {                     // far from the usual size: scaled anew, from the codebook itself
        const float* cb = kKeys ? a.key_cb + static_cast<long long>(h) * a.key_cb_stride
                                : a.val_cb + static_cast<long long>(h) * a.val_cb_stride;
        for (int i = tid; i < book_items<C, kWide>(held); i += 32 * kWarps) {
          const float4* x = reinterpret_cast<const float4*>(book_item<C, kWide>(cb, rounds, rank, i));
          sts16((kKeys ? cb_k : cb_v) + i * 16, scaled_halves(__ldg(x), __ldg(x + 1), pow2(e), kKeys));
        }
        asm volatile("bar.sync %0, %1;" ::"n"(kKeys ? 1 : 2), "n"(32 * kWarps) : "memory");
      }
      Phase step;
      if (kKeys && !kWide) step.get(steps);       // 64-scalar groups have no registers for it
      // rounds beyond the held ones: this thread's 16 bytes of every codeword, in fp16 and in fp32
      const unsigned char* far_book = static_cast<const unsigned char*>(a.book) +
                                      ((static_cast<size_t>(h) * C + rank) * 2 + (kKeys ? 0 : 1)) * (static_cast<size_t>(rounds) * kWideCodes * 128) + cl * 16;
      const float* far_cb = (kKeys ? a.key_cb + static_cast<long long>(h) * a.key_cb_stride : a.val_cb + static_cast<long long>(h) * a.val_cb_stride) +
                            static_cast<size_t>(rank) * rounds * kWideCodes * 64 + cl * 8;
      constexpr int kUnroll = kWide ? 1 : 2;      // both stages, where the body is short
#pragma unroll kUnroll
      for (int i = 0; i < ntiles; ++i) {
        const int s = kStages == 2 ? i & 1 : 0, lap = i / kStages;
        auto stage_free = [&] { return lap == 0 || wait(empty + s, (lap - 1) & 1, a.fault); };
        const long long left = end - (start + static_cast<long long>(i) * kGroupTok);
        if (kKeys && i % kReanchor == 0 && i > 0) anchor(i);
        if constexpr (kWide) {
          uint32_t own[kWords];
#pragma unroll
          for (int k = 0; k < kWords; ++k) own[k] = __funnelshift_r(lo[k], hi[k], shift);
          // every round's word now where the registers allow it, else when it is used
          auto pass = [&](int r) { return __shfl_sync(0xffffffffu, own[r / 8], (lane & 24) | (r & 7)); };
          constexpr bool kNow = R <= kWideRoundsPerCta;
          uint32_t all[kNow ? R : 1];
#pragma unroll
          for (int r = 0; r < (kNow ? R : 0); ++r) all[r] = pass(r);
          auto word = [&](int r) { return kNow ? all[kNow ? r : 0] : pass(r); };
          auto codeword = [&](int r, uint32_t w, int u) {
            const uint32_t at = entry(w, u);
            if (r < kHeldRounds) return lds16(book + r * (kWideCodes * 128) + at);
            if (e == kUsualScale)
              return __ldg(reinterpret_cast<const uint4*>(far_book + r * (kWideCodes * 128) + at));
            const float4* x = reinterpret_cast<const float4*>(far_cb + (r * (kWideCodes * 128) + at) / 2);
            return scaled_halves(__ldg(x), __ldg(x + 1), pow2(e), kKeys);
          };
          if (i + 1 < ntiles) load_words(i + 1);      // own[] is taken
          if (!stage_free()) break;
#pragma unroll
          for (int u0 = 0; u0 < kPer; u0 += 2) {
            // the codewords of all rounds, summed: neighbouring rounds in fp16 (rounded once
            // more), those sums in fp32
            float x[2][8];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int d = 0; d < 8; ++d) x[u][d] = 0.f;
#pragma unroll
            for (int r = 0; r < R; r += 2) {
              if (r >= rounds) continue;
              const int r1 = r + 1 < R ? r + 1 : r;
              const bool both = r1 > r && r1 < rounds;
              const uint32_t w0 = word(r), w1 = word(r1);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint4 y = codeword(r, w0, u0 + u);
                if (both) y = add_chunks(y, codeword(r1, w1, u0 + u));
                add_chunk(x[u], y);
              }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (kKeys) {
                store(s, u0 + u, ph.rotate(x[u]));
                Phase w;
                w.get(u0 + u < kPer - 1 ? steps : jumps);
                ph.turn(w);
              } else {
                uint4 v = make_uint4(half_pair(x[u][0], x[u][1]), half_pair(x[u][2], x[u][3]), half_pair(x[u][4], x[u][5]),
                                     half_pair(x[u][6], x[u][7]));
                if (token(u0 + u) >= left) v = make_uint4(0u, 0u, 0u, 0u);  // weight 0 times this must be 0
                store(s, u0 + u, v);
              }
            }
          }
        } else {
          uint64_t* c_full = &ctl.c_full[kKeys ? 0 : 1][i % kCodeStages];
          if (!wait(c_full, (i / kCodeStages) & 1, a.fault)) break;
          uint32_t codes_of[kPer * R];
#pragma unroll
          for (int j = 0; j < kPer * R; ++j) codes_of[j] = code(i, j / R, j % R);
          constexpr int kBatch = kPer < 4 ? kPer : 4;                        // gathers in flight
          bool ok = true;
#pragma unroll
          for (int u0 = 0; u0 < kPer; u0 += kBatch) {
            uint4 v[kBatch * R];
#pragma unroll
            for (int j = 0; j < kBatch * R; ++j) v[j] = lds16(book + (j % R) * (kCodes * CH * 16) + codes_of[u0 * R + j] * (CH * 16));
            if (u0 == 0) ok = stage_free();
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              uint4 x = v[u * R];
#pragma unroll
              for (int r = 1; r < R; ++r) x = add_chunks(x, v[u * R + r]);
              if (kKeys) {
                x = ph.rotate(x);
                ph.turn(step);
              } else if (left < kGroupTok && token(u0 + u) >= left) {
                x = make_uint4(0u, 0u, 0u, 0u);
              }
              store(s, u0 + u, x);
            }
          }
          if (!ok) break;
        }
        publish(s);
        if (!kWide && lane == 0) arrive(&ctl.c_empty[kKeys ? 0 : 1][i % kCodeStages]);
      }
    };
    if (warp < W::kValueWarp) produce(std::true_type{});
    else produce(std::false_type{});
  } else if (warp == kCopyWarp) {
    // ================= codes =================
    if (lane == 0) {
      const size_t row = static_cast<size_t>(R) * kGroups;
      auto copy_codes = [&](int i, int values) {
        const int s = i % kCodeStages;
        uint64_t* full = &ctl.c_full[values][s];
        if (i >= kCodeStages && !wait(&ctl.c_empty[values][s], (i / kCodeStages - 1) & 1, a.fault)) return false;
        const long long t = start + static_cast<long long>(i) * kGroupTok;
        const uint32_t bytes = static_cast<uint32_t>(min(end - t, static_cast<long long>(kGroupTok))) * static_cast<uint32_t>(row);
        mbar_expect_tx(full, bytes);
        bulk_load(smem + (ring - tiles_k) + s * (2 * kCodeBytes) + values * kCodeBytes,
                  (values ? a.val_codes : a.key_codes) + (static_cast<size_t>(h) * a.t_cap + t) * row, bytes, full);
        return true;
      };
      const int first = kWide ? 0 : min(ntiles, kCodeStages);
      for (int i = 0; i < first; ++i) {
        copy_codes(i, 0);
        copy_codes(i, 1);
      }
      asm volatile("griddepcontrol.wait;" ::: "memory");
      constexpr uint32_t kPiece = 16384;
      mbar_expect_tx(&ctl.book, 2 * cb_bytes);
      const uint32_t stored = kWide ? rounds * kWideCodes * 128 : cb_bytes;   // of keys or values in the workspace
      const unsigned char* book = static_cast<const unsigned char*>(a.book) + (static_cast<size_t>(h) * C + rank) * (2 * static_cast<size_t>(stored));
      for (uint32_t side = 0; side < 2; ++side)
        for (uint32_t at = 0; at < cb_bytes; at += kPiece)
          bulk_load(smem + (cb_k - tiles_k) + side * cb_bytes + at, book + side * stored + at, min(kPiece, cb_bytes - at), &ctl.book);
      if (!kWide) {
        bool ok = true;
        for (int i = first; ok && i < ntiles + 2; ++i) {                   // values are two steps behind
          if (i < ntiles) ok = copy_codes(i, 0);
          if (ok && i - 2 >= first) ok = copy_codes(i - 2, 1);
        }
        // no copy is left in flight, whatever ended the others' loops
        for (int i = max(0, ntiles - kCodeStages); ok && i < ntiles; ++i)
          ok = wait(&ctl.c_full[0][i % kCodeStages], (i / kCodeStages) & 1, a.fault) &&
               wait(&ctl.c_full[1][i % kCodeStages], (i / kCodeStages) & 1, a.fault);
      }
      wait(&ctl.book, 0, a.fault);
    }
  } else if (elect_one()) {
    // ================= matrix products =================
    // A tile is two halves of 64 dims, each [64 tokens][128 bytes] with 16-byte chunk c of row t
    // at c ^ (t & 7).  As keys (N = tokens, K = dims, K-major) 8 rows are 1024 bytes apart and 16
    // dims 32 bytes; as values (N = dims, K = tokens, N-major) 64 dims are a half apart and 8
    // tokens 1024 bytes.  Scores and outputs are issued by a warp each: the waits and issue of
    // both in one took longer than the products.
    constexpr uint32_t kDescS = (1u << 4) | ((kTok >> 3) << 17) | ((kRows >> 4) << 24);
    constexpr uint32_t kDescO = (1u << 4) | (1u << 16) | ((kHeadDim >> 3) << 17) | ((kRows >> 4) << 24);
    if (warp == kScoreWarp) {
      bool ok = wait(&ctl.q_full, 0, a.fault);
      for (int i = 0; ok && i < ntiles; ++i) {
        const int u = i & 1;
        ok = wait(&ctl.k_full[u], (i >> 1) & 1, a.fault) && (i < 2 || wait(&ctl.s_empty[u], ((i >> 1) - 1) & 1, a.fault));
        if (!ok) break;
        if (C == 2) fence_proxy_async_smem();     // the other CTA's stores
        tmem_after_sync();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_f16(tmem + kColS + u * kTok, tmem + kColQ + 8 * k,
                  operand(tiles_k + u * kTile + (k >> 2) * kHalfTile + (k & 3) * 32, 16, 1024), kDescS, k > 0);
        commit<C>(&ctl.s_full[u], false);
        if (i + 2 < ntiles) commit<C>(&ctl.k_empty[u], true);
      }
    } else {
      for (int i = 0; i < ntiles; ++i) {
        const int u = i & 1, s = kVStages == 2 ? u : 0;
        if (!wait(&ctl.v_full[s], (i / kVStages) & 1, a.fault) || !wait(&ctl.p_full[u], (i >> 1) & 1, a.fault)) break;
        if (C == 2) fence_proxy_async_smem();
        tmem_after_sync();
#pragma unroll
        for (int k = 0; k < kTok / 16; ++k)
          mma_f16(tmem + kColO + u * kHeadDim, tmem + kColP + u * 32 + 8 * k,
                  operand(tiles_v + s * kTile + k * 2048, kHalfTile, 1024), kDescO, i >= 2 || k > 0);
        if (i + kVStages < ntiles) commit<C>(&ctl.v_empty[s], true);
        commit<C>(&ctl.pv_done[u], false);
      }
    }
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();                                // tiles and codebooks are no longer read

  // ---- join the two streams and write this CTA's partial state ----
  // Stream st finishes the dims 64 st .. 64 st + 63 and leaves its others to the other stream.
  float* rows_out = reinterpret_cast<float*>(smem);
  const int st = warp >> 2, r = (warp & 3) * 32 + lane;
  const bool joins = warp < kSoftWarps && (warp & 3) < nact, have = st == 0 || ntiles > 1;
  const uint32_t out_cols = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO + (st & 1) * kHeadDim;
  if (joins) {
    ctl.m[st][r] = m;
    ctl.l[st][r] = l;
#pragma unroll 1
    for (int c = 64 * (1 - st); c < 64 * (2 - st); c += 32) {
      uint32_t o[32];
      tmem_load32(o, out_cols + c);
      tmem_load_wait();
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<uint4*>(rows_out + r * kOutPitch + c + j) =
            have ? make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncthreads();
  if (joins) {
    const float m1 = ctl.m[1 - st][r], l1 = ctl.l[1 - st][r];
    const float M = fmaxf(m, m1), ref = M == -INFINITY ? 0.f : M;
    const float back = pow2(-ev), f0 = exp2f(m - ref), f1 = exp2f(m1 - ref);
#pragma unroll 1
    for (int c = 64 * st; c < 64 * (st + 1); c += 32) {
      uint32_t o[32];
      tmem_load32(o, out_cols + c);
      tmem_load_wait();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        float4* at = reinterpret_cast<float4*>(rows_out + r * kOutPitch + c + j);
        float4 x = *at;
        x = make_float4(x.x * f1, x.y * f1, x.z * f1, x.w * f1);
        if (have) {
          x.x = fmaf(__uint_as_float(o[j]), f0, x.x);
          x.y = fmaf(__uint_as_float(o[j + 1]), f0, x.y);
          x.z = fmaf(__uint_as_float(o[j + 2]), f0, x.z);
          x.w = fmaf(__uint_as_float(o[j + 3]), f0, x.w);
        }
        *at = make_float4(x.x * back, x.y * back, x.z * back, x.w * back);
      }
    }
    if (st == 0 && r < nrows) {
      const size_t at = global_row(r) * n_parts + blockIdx.x;
      a.part_m[at] = M;
      a.part_l[at] = fmaf(l, f0, l1 * f1);
    }
  }
  tmem_before_sync();
  __syncthreads();
  for (int i = threadIdx.x; i < nrows * 32; i += kThreads) {
    const int rr = i >> 5, c = (i & 31) * 4;
    *reinterpret_cast<float4*>(a.part_o + (global_row(rr) * n_parts + blockIdx.x) * kHeadDim + c) =
        *reinterpret_cast<const float4*>(rows_out + rr * kOutPitch + c);
  }
  if (warp == kScoreWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  if (C == 2) cluster_barrier();                  // the other CTA may still store here until now
}

template <int C, bool kWide, int R>
cudaError_t run(const ServeArgs& a, cudaStream_t stream) {
  static PerDeviceFlag flag;
  constexpr int kTiles = (kWide ? 3 : 4) * kTile;
  constexpr size_t kCodes8 = kWide ? 0 : kMostCodeStages / C * 2 * C * kTok * R * kGroups;
  constexpr size_t kMost = kTiles + 32 * book_items<C, kWide>(held_rounds<kWide>(R)) + kCodes8 + sizeof(Control);
  static_assert(kMost <= 227 * 1024, "fits an SM");
  cudaError_t e = set_smem_limit_once(flag, prefix_mma_kernel<C, kWide, R>, kMost);
  if (e != cudaSuccess) return e;
  e = launch_chained(prefix_book_kernel<C, kWide>, dim3(book_items<C, kWide>(a.R) / kBookThreads, 2 * C, a.n_kv_heads), kBookThreads, a, stream);
  if (e != cudaSuccess) return e;
  size_t bytes = kTiles + 32 * static_cast<size_t>(book_items<C, kWide>(held_rounds<kWide>(a.R))) + kCodes8;
  if (bytes < kOutBytes) bytes = kOutBytes;
  bytes += sizeof(Control);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_splits * C, a.n_kv_heads, (a.batch * a.group + kRows - 1) / kRows);
  cfg.blockDim = dim3(Roles<kWide>::kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, prefix_mma_kernel<C, kWide, R>, a);
}

}  // namespace

cudaError_t launch_prefix_mma(const ServeArgs& a, cudaStream_t stream) {
  if (a.wide) return a.R <= kWideRoundsPerCta ? run<2, true, kWideRoundsPerCta>(a, stream) : run<2, true, kWideMaxR>(a, stream);
  return a.R == 1 ? run<1, false, 1>(a, stream) : run<2, false, 2>(a, stream);
}

}  // namespace cvq
