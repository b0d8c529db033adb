// Shared-prefix attention of 16-bit queries on the tensor cores: each cached token is decoded
// from its codes once per KV head and block of 128 query rows, straight into the operand tiles of
// the matrix products, and read there by the query rows of every sequence.
//
// Precision: the products are fp16, of operands in two parts -- a decoded number x is held as
// hi = fp16(x) and lo = fp16(x - hi), 22 bits, and so are the softmax weights p; 16-bit queries are
// one fp16 number each, exactly.  S = Q (Khi + Klo)^T, and O sums Phi Vhi, Phi Vlo and Plo Vhi, which
// leaves out 2^-22 of a product.  Codewords, the sum of the rounds, the rotation and the phases are
// fp32, as are the sums of products, the softmax, O and the merge.  Codebooks and query rows are
// scaled by powers of two into fp16's range.
//
// A cluster of C CTAs shares 128 query rows ((sequence, head of the group) pairs) of a KV head and a
// run of tokens, in tiles of 64 tokens a CTA:
//   producers (8 warps for keys, 4 or 8 for values)  gather codewords from fp32 codebooks in
//                        shared memory, sum the rounds, rotate the keys and store the tiles
//   one thread           copies codes, steps ahead, into shared memory
//   two threads          S = Q K^T (M = 128 rows, N = 64 tokens; Q from TMEM), O += P V
//                        (N = 128 dims; P from TMEM, over the scores), both tcgen05.mma kind::f16
//   softmax (2 x 4 warps)  a thread owns a row: even tiles go to the first four warps, odd
//                        ones to the others, each with its own O, maximum and sum (joined at
//                        the end), so that the exponentials of one tile run under the other's
//                        loads and barriers
//
// Split over the cluster: fp32 codebooks of one round of 8-scalar groups fill two SMs, of two
// rounds or of 64-scalar groups four.  So a CTA holds the codebooks of 128 / C dims, decodes these of
// all the cluster's tokens and stores the others' tiles through distributed shared memory (st.async,
// whose bytes the receiver's barrier counts, so that nothing waits for them at the sender).  Rounds of
// 64-scalar groups that do not fit (beyond 9) are gathered from the codebooks themselves.
//
// Bank conflicts: codebooks lie as [round][code][quad of 4 dims], so the 8 lanes that work on the quads
// of one token read 8 different bank groups whatever their codes are.
//
// Phases: a producer thread keeps e^{i theta t} of its 2 pairs in fp32 and turns them on from
// token to token, 15 times at most before they are taken anew from the exact turns: each turn adds
// an error of 2^-24, and the step's own rounding once more.
//
// What bounds it: the producers (fp32 sums, rotation, two parts of every number) and the products, 2.5
// times those of one part, whose tiles have one stage: two would not fit beside the codebooks.
// Measured in a captured graph, 32 query and 8 KV heads: 32 sequences over 131072 tokens, R = 1, 271 us
// (2.5 times 68.7 GF: 630 TFLOP/s); 16 over 32768, R = 2, 93 us, and R = 11 of 64-scalar groups
// 218 us; a short prefix 16 us, of which the codebooks' order takes 3 and the join and merge 4.  Operands
// of one part took 103, 42, 111 and 12 us, with outputs 3e-4 off instead of 3e-6 and lse 1e-6 instead of
// 5e-8.
#include <type_traits>

#include "serve.cuh"

namespace cvq {

namespace {

constexpr int kSoftWarps = 8;
// The warps by their roles.
template <bool kWide>
struct Roles {
  static constexpr int kKeyWarps = 8, kValueWarps = 8;
  static constexpr int kValueWarp = kSoftWarps + kKeyWarps;                   // the first
  static constexpr int kScoreWarp = kValueWarp + kValueWarps, kOutWarp = kScoreWarp + 1, kCopyWarp = kOutWarp + 1;
  static constexpr int kThreads = 32 * (kCopyWarp + 1);
};
constexpr int kRows = 128;
constexpr int kHalfTile = kTok * 128;             // 64 dims of one part of its keys or values, bytes
constexpr int kTile = 2 * kHalfTile;              // one part; the second follows
constexpr int kMostCodeStages = 4;
constexpr int kReanchor = 2;                      // steps between exact phases
constexpr int kOutPitch = kHeadDim + 4;           // floats; 16-byte chunks of 8 rows in 8 bank groups
constexpr int kOutBytes = kRows * kOutPitch * 4;
// columns of TMEM: S of the two streams (and over each, 32 scores at a time, the two parts of their
// weights), Q, their O
constexpr uint32_t kColS = 0, kColQ = 128, kColO = 256, kTmemCols = 512;

struct Control {
  uint64_t book;                                  // codebooks
  uint64_t q_full;
  uint64_t c_full[2][kMostCodeStages], c_empty[2][kMostCodeStages];         // codes of keys, values
  uint64_t k_full, k_empty, v_full, v_empty, s_full[2], p_full[2], pv_done[2];
  uint32_t tmem;
  alignas(16) float turn[2][16][4];               // steps and jumps of the phases, per quad
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
__device__ __forceinline__ void commit(uint64_t* bar, bool all) {
  if (all) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>((1 << C) - 1)) : "memory");
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
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
// to another CTA; its barrier counts the bytes as they land, so that nothing waits for them here
__device__ __forceinline__ void send8(uint32_t addr, uint32_t x, uint32_t y, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1,%2}, [%3];" ::"r"(addr), "r"(x), "r"(y),
               "r"(bar) : "memory");
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
// a pair of numbers as the nearest fp16 numbers, and what they leave out in `rest`
__device__ __forceinline__ uint32_t take_half(f2 x, uint32_t& rest) {
  const float2 v = unpack(x);
  const uint32_t h = half_pair(v.x, v.y);
  const float2 near = floats_of(h);
  const float2 left = unpack(add2(x, neg2(pack(near.x, near.y))));
  rest = half_pair(left.x, left.y);
  return h;
}
// adds to memory that no other thread touches meanwhile
__device__ __forceinline__ void add_global(float4* at, float4 v) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1,%2,%3,%4};" ::"l"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t lds4(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// e^{i theta_j t} of the 2 pairs of a quad, times a power of two
struct Phase {
  f2 c, s;
  __device__ __forceinline__ void set(const PhaseTurns& ph, int quad, unsigned long long t, float scale) {
    const float2 u = phase_exact(ph.F[2 * quad] * t), v = phase_exact(ph.F[2 * quad + 1] * t);
    c = pack(u.x * scale, v.x * scale);
    s = pack(u.y * scale, v.y * scale);
  }
  __device__ __forceinline__ void put(float* at) const {
    const float2 x = unpack(c), y = unpack(s);
    *reinterpret_cast<float4*>(at) = make_float4(x.x, x.y, y.x, y.y);
  }
  __device__ __forceinline__ void get(const float* at) {
    const float4 x = *reinterpret_cast<const float4*>(at);
    c = pack(x.x, x.y);
    s = pack(x.z, x.w);
  }
  __device__ __forceinline__ void turn(const Phase& w) {
    const f2 nc = fma2(neg2(s), w.s, mul2(c, w.c));
    s = fma2(s, w.c, mul2(c, w.s));
    c = nc;
  }
  // the real (re) and imaginary parts (im) of two pairs, turned
  __device__ __forceinline__ void rotate(f2& re, f2& im) const {
    const f2 a = fma2(im, neg2(s), mul2(re, c));
    im = fma2(im, c, mul2(re, s));
    re = a;
  }
};

// ---- codebooks ----
// CTA `rank` of a cluster of C holds dims 128 / C * rank on, in quads of 4: NQ = 32 / C of them.
// Items of 16 bytes lie as [round][entry][quad].  Keys are held, here and in the operand tiles, with
// the two real and the two imaginary parts of two pairs side by side, so that two pairs rotate at once.
template <int C, bool kWide>
__host__ __device__ constexpr int book_items(int R) {
  return R * (kWide ? kWideCodes : kCodes) * (32 / C);
}
// where item (round r, entry, quad) of a KV head's codebook comes from
template <bool kWide>
__device__ __forceinline__ const float* book_item(const float* cb, int R, int r, int entry, int quad) {
  if (kWide)
    return cb + ((static_cast<size_t>(quad >> 4) * R + r) * kWideCodes + entry) * kWideGroupDim + (quad & 15) * 4;
  return cb + ((static_cast<size_t>(quad >> 1) * R + r) * kCodes + entry) * kCodeword + (quad & 1) * 4;
}
// rounds of 64-scalar groups that fit in shared memory beside R rounds of codes
__host__ __device__ constexpr int held_rounds(int R) { return R <= 9 ? R : R <= 11 ? 9 : 8; }

constexpr int kBookThreads = 256;

// The codebooks in the order in which CTAs of the attention kernel hold them, into the workspace, and
// the largest finite |x| of every 256 items: once a call, so that a CTA copies its share in one
// piece.  Launched before the attention kernel, whose own set-up runs under it.
template <int C, bool kWide>
__global__ void __launch_bounds__(kBookThreads) prefix_book_kernel(const __grid_constant__ ServeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");                        // for what ran before this call
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t warp_peak[kBookThreads / 32];
  constexpr int NQ = 32 / C, kEntries = kWide ? kWideCodes : kCodes;
  const int n = book_items<C, kWide>(a.R), i = blockIdx.x * kBookThreads + threadIdx.x;
  const int rank = blockIdx.y >> 1, values = blockIdx.y & 1, h = blockIdx.z;
  const float* cb = values ? a.val_cb + static_cast<long long>(h) * a.val_cb_stride
                           : a.key_cb + static_cast<long long>(h) * a.key_cb_stride;
  float4 x = __ldg(reinterpret_cast<const float4*>(book_item<kWide>(cb, a.R, i / (NQ * kEntries), i / NQ % kEntries, rank * NQ + i % NQ)));
  const float v[4] = {x.x, x.y, x.z, x.w};
  uint32_t peak = 0;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t bits = __float_as_uint(v[d]) & 0x7fffffffu;
    if (bits < 0x7f800000u) peak = max(peak, bits);
  }
  if (!values) x = make_float4(v[0], v[2], v[1], v[3]);
  if (in_bounds(a.fault, i, n)) reinterpret_cast<float4*>(a.book)[((static_cast<size_t>(h) * C + rank) * 2 + values) * n + i] = x;
  peak = __reduce_max_sync(0xffffffffu, peak);
  if ((threadIdx.x & 31) == 0) warp_peak[threadIdx.x >> 5] = peak;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kBookThreads / 32; ++w) peak = max(peak, warp_peak[w]);
    a.book_peak[((static_cast<size_t>(h) * 2 + values) * C + rank) * gridDim.x + blockIdx.x] = peak;
  }
}
// Exponent of the scale that brings sums of R codewords of at most `peak`, rotated, below 2^15.
__device__ __forceinline__ int scale_exponent(uint32_t peak_bits, int R) {
  if (peak_bits == 0) return 0;
  const int grow = 32 - __clz(2 * R - 1);         // 2^grow >= 2 R > sqrt(2) R
  return min(max(14 - log2_floor(__uint_as_float(peak_bits)) - grow, -126), 120);
}

// two 16-bit query elements as floats
__device__ __forceinline__ float2 query_pair(uint32_t w, bool bf16) {
  return bf16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : floats_of(w);
}

// The layout of shared memory behind the tiles: codebooks of keys and values, the ring of codes.
template <int C, bool kWide, int R>
struct Layout {
  static constexpr int kGroupTok = C * kTok;      // tokens of a step of the cluster
  static constexpr int kCodeStages = kWide || R == 2 ? 2 : 4;
  // codes of 64-scalar groups: a row per round, 16 bytes apart in banks
  static constexpr int kPitch = kGroupTok + 16;
  // one codebook, and a stage of one side's codes (8-scalar groups: [token][round][16], as in the cache)
  static __host__ __device__ constexpr uint32_t book(int rounds) { return 16u * book_items<C, kWide>(kWide ? held_rounds(rounds) : R); }
  static __host__ __device__ constexpr uint32_t codes(int rounds) { return kWide ? rounds * kPitch : kGroupTok * R * kGroups; }
  static __host__ __device__ constexpr uint32_t control(int rounds) { return 4 * kTile + 2 * book(rounds) + 2 * kCodeStages * codes(rounds); }
  static __host__ __device__ constexpr uint32_t bytes(int rounds) { return control(rounds) + sizeof(Control); }
};

// R: rounds of 8-scalar groups; 64-scalar groups (kWide) take a.R
template <int C, bool kWide, int R>
__global__ void __launch_bounds__(Roles<kWide>::kThreads, 1) prefix_mma_kernel(const __grid_constant__ ServeArgs a) {
  using W = Roles<kWide>;
  using Lay = Layout<C, kWide, R>;
  constexpr int kThreads = W::kThreads, kScoreWarp = W::kScoreWarp, kCopyWarp = W::kCopyWarp;
  constexpr int kGroupTok = Lay::kGroupTok, kCodeStages = Lay::kCodeStages, NQ = 32 / C;
  static_assert(C == (kWide ? 4 : 2 * R), "a CTA's dims");
  extern __shared__ __align__(1024) unsigned char smem[];
  const int rounds = kWide ? a.R : R;
  const uint32_t tiles_k = smem_u32(smem), tiles_v = tiles_k + 2 * kTile, cb_k = tiles_v + 2 * kTile;
  const uint32_t cb_bytes = Lay::book(rounds), cb_v = cb_k + cb_bytes;
  const uint32_t code_bytes = Lay::codes(rounds), ring = cb_v + cb_bytes;    // a stage: keys, then values
  Control& ctl = *reinterpret_cast<Control*>(smem + Lay::control(rounds));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x % C);
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
  const long long per = ((static_cast<long long>(L) + a.n_splits - 1) / a.n_splits + kGroupTok - 1) / kGroupTok * kGroupTok;
  const long long start = min(per * split, static_cast<long long>(L)), end = min(start + per, static_cast<long long>(L));
  const int ntiles = static_cast<int>((end - start + kGroupTok - 1) / kGroupTok);
  if (ntiles == 0) {                              // the same for all CTAs of a cluster
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x < nrows) {
      const size_t at = global_row(threadIdx.x) * n_parts + blockIdx.x;
      if (in_bounds(a.fault, at, n_part_rows(a))) {
        a.part_m[at] = -INFINITY;
        a.part_l[at] = 0.f;
      }
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
    mbar_init(&ctl.k_full, W::kKeyWarps);
    mbar_init(&ctl.v_full, W::kValueWarps);
    mbar_init(&ctl.k_empty, C);
    mbar_init(&ctl.v_empty, C);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.s_full[s], 1);
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
  cluster_barrier();                              // the other CTAs run, and their barriers are there
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
  // The matrix instructions cut their sums off instead of rounding them, so a long O comes out too
  // small (by 1e-4 after 1024 tiles).  Every kFlush tiles of a stream its O is therefore added, in
  // fp32 and relative to the maximum m_kept, to the workspace, and begun anew.
  float m_kept = -INFINITY;
  auto kept_row = [&](int stream, int r) {
    const size_t at = global_row(min(r, nrows - 1)) * n_parts + blockIdx.x;
    return reinterpret_cast<float4*>(a.kept_o + ((in_bounds(a.fault, at, n_part_rows(a)) ? at : 0) * 2 + stream) * kHeadDim);
  };
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
      // Scores of the operands are below 2^31: a factor of 2^-123 makes them all nothing, and a
      // smaller one would underflow to 0, which turns the -inf of masked scores into NaN
      const int by = min(max(-eq - e.x, -120), 252);
      const float factor = 0.08838834764831845f * kLog2e * pow2(by / 2) * pow2(by - by / 2);
      auto flush = [&](bool first) {
        float4* to = kept_row(st, q4 * 32 + lane);
        const bool mine = q4 * 32 + lane < nrows, moved = __any_sync(0xffffffffu, m != m_kept);
        const float f = m == m_kept ? 1.f : exp2f(m_kept - m);
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 16) {
          uint32_t o[16];
          tmem_load16(o, lanes + kColO + st * kHeadDim + c);
          tmem_load_wait();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float4 x = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]), __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
            float4* at = to + c / 4 + j;
            if (!mine) continue;
            if (first || moved) {
              if (!first) {
                const float4 y = __ldcg(at);
                x = make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
              }
              __stcg(at, x);
            } else {
              add_global(at, x);
            }
          }
        }
        m_kept = m;
      };
      for (int i = st; i < ntiles; i += 2) {
        const unsigned par = (i >> 1) & 1;
        if (!wait(&ctl.s_full[st], par, a.fault)) break;
        tmem_after_sync();
        const bool fresh = (i >> 1) % kFlush == 0;                          // O starts with this tile
        if (i >= 2 && fresh) {
          if (!wait(&ctl.pv_done[st], par ^ 1, a.fault)) break;
          tmem_after_sync();
          flush((i >> 1) == kFlush);
        }
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
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 1; c >= 0; --c) {
          load_scores(c, s[c % kHeld]);
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            mx4[j / 2 & 3] = fmaxf(mx4[j / 2 & 3], fmaxf(__uint_as_float(s[c % kHeld][j]), __uint_as_float(s[c % kHeld][j + 1])));
        }
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        mx *= factor;
        const bool grow = mx > m + kSlack || (m == -INFINITY && mx > m);
        const float alpha = grow ? exp2f(m - mx) : 1.f;
        if (grow) m = mx;
        const float ref = m == -INFINITY ? 0.f : m - kLift;
        const f2 ff = pack(factor, factor), rr = pack(-ref, -ref);
        // these scores came after the stream's last weights had been used, which lay in their place
        if (!fresh && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!wait(&ctl.pv_done[st], par ^ 1, a.fault)) break;
          tmem_after_sync();
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
        f2 sum = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {             // 16 weights, their two parts
          if (kHeld == 1 && c == 2) load_scores(1, s[0]);
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t(&x)[32] = s[c / 2 % kHeld];
            const int k = 16 * (c & 1) + 2 * j;
            const float2 y = unpack(fma2(pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), ff, rr));
            const f2 e01 = pack(exp2_fast(y.x), exp2_fast(y.y));
            sum = add2(sum, e01);
            hi[j] = take_half(e01, lo[j]);
          }
          tmem_store8(lanes + kColS + st * kTok + 32 * (c >> 1) + 8 * (c & 1), hi);
          tmem_store8(lanes + kColS + st * kTok + 32 * (c >> 1) + 8 * (c & 1) + 16, lo);
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
    m_kept -= kLift;
    if (m != -INFINITY) m -= kLift;
  } else if (warp < kScoreWarp) {
    // ================= producers =================
    // Keys and values are made by warps of their own; a thread makes one quad of dims.
    auto produce = [&](auto is_keys) {
      constexpr bool kKeys = decltype(is_keys)::value;
      constexpr int kWarps = kKeys ? W::kKeyWarps : W::kValueWarps, kFirst = kKeys ? kSoftWarps : W::kValueWarp;
      constexpr int kSlots = 32 * kWarps / NQ;    // threads of a quad
      // tokens that a thread takes one after another (codes of 64-scalar groups: 4 to a word), and how
      // often in a step
      constexpr int kRun = kWide ? 4 : 1, kPasses = kGroupTok / (kSlots * kRun);
      static_assert(kSlots % 8 == 0 && (kWide ? kSlots * kRun == 2 * kTok : kTok % kSlots == 0), "rows of a thread");
      const int tid = threadIdx.x - 32 * kFirst, q = tid % NQ, slot = tid / NQ;
      const int quad = rank * NQ + q, chunk = quad >> 1;
      uint64_t* full = kKeys ? &ctl.k_full : &ctl.v_full;
      uint64_t* empty = kKeys ? &ctl.k_empty : &ctl.v_empty;
      const uint32_t book = (kKeys ? cb_k : cb_v) + q * 16;
      // Token u of pass p within a step lies in row token % 64 of CTA token / 64: 8 bytes of each part.
      auto token = [&](int p, int u) { return (p * kSlots + slot) * kRun + u; };
      const int row = token(0, 0) % kTok;
      const uint32_t at0 = (kKeys ? tiles_k : tiles_v) + (chunk >> 3) * kHalfTile + row * 128 + (q & 1) * 8;
      const uint32_t swizzle = (chunk & 7) ^ (row & 7);
      auto store = [&](int p, int u, f2 x, f2 y) {
        uint32_t l0, l1;
        const uint32_t h0 = take_half(x, l0), h1 = take_half(y, l1);
        const uint32_t tile = kKeys ? tiles_k : tiles_v;
        uint32_t at = at0 + (kWide ? u * 128 + ((swizzle ^ u) << 4) : (p * kSlots % kTok) * 128 + (swizzle << 4));
        uint32_t to = kWide ? 2 * p + slot / (kTok / kRun) : p * kSlots / kTok;
        // debug build: bytes that others wait for go to a place that there is
        if (!in_bounds(a.fault, at - tile + 7, kTile)) at = tile;
        if (!in_bounds(a.fault, to, C)) to = rank;
        if (to == static_cast<uint32_t>(rank)) {
          sts8(at, h0, h1);
          sts8(at + kTile, l0, l1);
        } else {
          const uint32_t away = map_to(at, to), bar = map_to(smem_u32(full), to);
          send8(away, h0, h1, bar);
          send8(away + kTile, l0, l1, bar);
        }
      };
      // a tile is full when this CTA's warps have stored and the others' shares have landed
      auto publish = [&] {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (warp == kFirst) mbar_expect_tx(full, 2 * kTile / C * (C - 1));
          else arrive(full);
        }
      };
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const int2 both = book_exponents();
      const float scale = pow2(kKeys ? both.x : both.y);
      // phases: this thread's own in registers, what they turn by from token to token (and from pass to
      // pass) in shared memory, where a quad's threads share it
      Phase ph;
      if (kKeys) {
        if (slot < (kWide ? 2 : 1)) {
          ph.set(a.phase, quad, kWide ? (slot == 0 ? 1 : kSlots * kRun - (kRun - 1)) : kSlots, 1.f);
          ph.put(ctl.turn[slot][q]);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      }
      auto anchor = [&](int i) {
        ph.set(a.phase, quad, static_cast<unsigned long long>(start + static_cast<long long>(i) * kGroupTok + token(0, 0)), scale);
      };
      const f2 scale2 = pack(scale, scale);
      Phase step;
      if (kKeys && !kWide) step.get(ctl.turn[0][q]);
      wait(&ctl.book, 0, a.fault);
      const uint32_t codes = ring + (kKeys ? 0 : code_bytes);
      for (int i = 0; i < ntiles; ++i) {
        auto stage_free = [&] { return i == 0 || wait(empty, (i - 1) & 1, a.fault); };
        const long long left = end - (start + static_cast<long long>(i) * kGroupTok);
        if (kKeys && (kWide || i % kReanchor == 0)) anchor(i);
        if (!wait(&ctl.c_full[kKeys ? 0 : 1][i % kCodeStages], (i / kCodeStages) & 1, a.fault)) break;
        const uint32_t stage = codes + (i % kCodeStages) * (2 * code_bytes);
        bool ok = true;
        // one decoded quad of token (p, u): rotated, or scaled and, behind the last token, cleared (a
        // weight of 0 times it must be 0)
        auto finish = [&](int p, int u, f2 x, f2 y) {
          if (kKeys) {
            ph.rotate(x, y);
          } else {
            x = mul2(x, scale2);
            y = mul2(y, scale2);
            if (left < kGroupTok && token(p, u) >= left) x = y = 0;
          }
          store(p, u, x, y);
        };
        if constexpr (kWide) {
          const int held = held_rounds(rounds);
          const bool packed = a.code_bits == 6;
          const int unit = packed ? 6 : 8;
          const float* cb = kKeys ? a.key_cb + static_cast<long long>(h) * a.key_cb_stride : a.val_cb + static_cast<long long>(h) * a.val_cb_stride;
#pragma unroll 1
          for (int p = 0; p < kPasses; ++p) {
            // the codes of this thread's 4 tokens: 4 bytes of a round's row, or 3 anywhere in two words
            const uint32_t off = (p * kSlots + slot) * (packed ? 3 : 4);
            const uint32_t from = stage + (off & ~3u);
            auto word = [&](int r) {
              if (!in_bounds(a.fault, r * Lay::kPitch + (off & ~3u) + (packed ? 7 : 3), code_bytes)) return 0u;
              const uint32_t w = lds4(from + r * Lay::kPitch);
              return packed ? __funnelshift_r(w, lds4(from + r * Lay::kPitch + 4), 8 * (off & 3)) : w;
            };
            f2 x[kRun][2];
#pragma unroll
            for (int u = 0; u < kRun; ++u) x[u][0] = x[u][1] = 0;
#pragma unroll 1
            for (int r = 0; r < held; ++r) {
              const uint32_t w = word(r), at = book + r * (kWideCodes * NQ * 16);
#pragma unroll
              for (int u = 0; u < kRun; ++u) {
                const uint4 v = lds16(at + ((w >> (unit * u)) & 63u) * (NQ * 16));
                x[u][0] = add2(x[u][0], pack(__uint_as_float(v.x), __uint_as_float(v.y)));
                x[u][1] = add2(x[u][1], pack(__uint_as_float(v.z), __uint_as_float(v.w)));
              }
            }
            for (int r = held; r < rounds; ++r) {
              const uint32_t w = word(r);
              const float* at = book_item<true>(cb, rounds, r, 0, quad);
              float4 v[kRun];
#pragma unroll
              for (int u = 0; u < kRun; ++u) v[u] = __ldg(reinterpret_cast<const float4*>(at + ((w >> (unit * u)) & 63u) * kWideGroupDim));
#pragma unroll
              for (int u = 0; u < kRun; ++u) {
                x[u][0] = add2(x[u][0], kKeys ? pack(v[u].x, v[u].z) : pack(v[u].x, v[u].y));
                x[u][1] = add2(x[u][1], kKeys ? pack(v[u].y, v[u].w) : pack(v[u].z, v[u].w));
              }
            }
            if (p == 0) ok = stage_free();
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < kRun; ++u) {
              finish(p, u, x[u][0], x[u][1]);
              if (kKeys) {
                step.get(ctl.turn[u < kRun - 1 ? 0 : 1][q]);
                ph.turn(step);
              }
            }
          }
        } else {
          // codes of the next 4 tokens are loaded under this one's gathers (behind the last token any
          // byte, all of them entries)
          constexpr int kBatch = 4;
          const uint32_t my_codes = stage + slot * (R * kGroups) + chunk;
          uint32_t code[kBatch * R];
          auto load_codes = [&](int p0) {
#pragma unroll
            for (int j = 0; j < kBatch * R; ++j) code[j] = lds1(my_codes + (p0 + j / R) * (kSlots * R * kGroups) + j % R * kGroups);
          };
          load_codes(0);
#pragma unroll
          for (int p0 = 0; p0 < kPasses; p0 += kBatch) {
            uint4 v[kBatch * R];
#pragma unroll
            for (int j = 0; j < kBatch * R; ++j) v[j] = lds16(book + ((j % R) * kCodes + code[j]) * (NQ * 16));
            if (p0 + kBatch < kPasses) load_codes(p0 + kBatch);
            if (p0 == 0) ok = stage_free();
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              f2 x = pack(__uint_as_float(v[u * R].x), __uint_as_float(v[u * R].y));
              f2 y = pack(__uint_as_float(v[u * R].z), __uint_as_float(v[u * R].w));
#pragma unroll
              for (int r = 1; r < R; ++r) {
                x = add2(x, pack(__uint_as_float(v[u * R + r].x), __uint_as_float(v[u * R + r].y)));
                y = add2(y, pack(__uint_as_float(v[u * R + r].z), __uint_as_float(v[u * R + r].w)));
              }
              finish(p0 + u, 0, x, y);
              if (kKeys) ph.turn(step);
            }
          }
        }
        if (!ok) break;
        publish();
        if (lane == 0) arrive(&ctl.c_empty[kKeys ? 0 : 1][i % kCodeStages]);
      }
    };
    if (warp < W::kValueWarp) produce(std::true_type{});
    else produce(std::false_type{});
  } else if (warp == kCopyWarp) {
    // ================= codes =================
    if (lane == 0) {
      auto copy_codes = [&](int i, int values) {
        const int s = i % kCodeStages;
        uint64_t* full = &ctl.c_full[values][s];
        if (i >= kCodeStages && !wait(&ctl.c_empty[values][s], (i / kCodeStages - 1) & 1, a.fault)) return false;
        const long long t = start + static_cast<long long>(i) * kGroupTok;
        const int n = static_cast<int>(min(end - t, static_cast<long long>(kGroupTok)));
        // debug build: no copy where one would leave the cache, or its stage
        const bool fits = in_bounds(a.fault, t + n - 1, a.t_cap) && in_bounds(a.fault, (2 * s + values + 1) * code_bytes - 1, 2 * kCodeStages * code_bytes);
        unsigned char* to = smem + (ring - tiles_k) + (2 * s + values) * code_bytes;
        const uint8_t* codes = values ? a.val_codes : a.key_codes;
        if (kWide) {                              // whole pieces of 16 bytes: rows are, of either kind
          const bool packed = a.code_bits == 6;
          const size_t row = packed ? static_cast<size_t>(a.t_cap) / 4 * 3 : static_cast<size_t>(a.t_cap);
          const uint32_t bytes = packed ? (n + 63) / 64 * 48 : (n + 15) / 16 * 16;
          const uint8_t* from = codes + (static_cast<size_t>(h) * kWideGroups + rank / (C / 2)) * rounds * row + (packed ? t / 4 * 3 : t);
          mbar_expect_tx(full, fits ? bytes * rounds : 0);
          for (int r = 0; r < rounds && fits; ++r) bulk_load(to + r * Lay::kPitch, from + r * row, bytes, full);
        } else {
          constexpr uint32_t row = R * kGroups;
          mbar_expect_tx(full, fits ? n * row : 0);
          if (fits) bulk_load(to, codes + (static_cast<size_t>(h) * a.t_cap + t) * row, n * row, full);
        }
        return true;
      };
      const int first = min(ntiles, kCodeStages);
      for (int i = 0; i < first; ++i) {
        copy_codes(i, 0);
        copy_codes(i, 1);
      }
      asm volatile("griddepcontrol.wait;" ::: "memory");
      constexpr uint32_t kPiece = 16384;
      mbar_expect_tx(&ctl.book, 2 * cb_bytes);
      const size_t stored = 16 * static_cast<size_t>(book_items<C, kWide>(rounds));   // of keys or values in the workspace
      const unsigned char* book = static_cast<const unsigned char*>(a.book) + (static_cast<size_t>(h) * C + rank) * (2 * stored);
      for (uint32_t side = 0; side < 2; ++side)
        for (uint32_t at = 0; at < cb_bytes; at += kPiece)
          bulk_load(smem + (cb_k - tiles_k) + side * cb_bytes + at, book + side * stored + at, min(kPiece, cb_bytes - at), &ctl.book);
      constexpr int kLate = kCodeStages / 2;      // steps that values are behind
      bool ok = true;
      for (int i = first; ok && i < ntiles + kLate; ++i) {
        if (i < ntiles) ok = copy_codes(i, 0);
        if (ok && i - kLate >= first) ok = copy_codes(i - kLate, 1);
      }
      // no copy is left in flight, whatever ended the others' loops
      for (int i = max(0, ntiles - kCodeStages); ok && i < ntiles; ++i)
        ok = wait(&ctl.c_full[0][i % kCodeStages], (i / kCodeStages) & 1, a.fault) &&
             wait(&ctl.c_full[1][i % kCodeStages], (i / kCodeStages) & 1, a.fault);
      wait(&ctl.book, 0, a.fault);
    }
  } else if (elect_one()) {
    // ================= matrix products =================
    // A part of a tile is two halves of 64 dims, each [64 tokens][128 bytes] with 16-byte chunk c of
    // row t at c ^ (t & 7).  As keys (N = tokens, K = dims, K-major) 8 rows are 1024 bytes apart and 16
    // dims 32 bytes; as values (N = dims, K = tokens, N-major) 64 dims are a half apart and 8
    // tokens 1024 bytes.  Scores and outputs are issued by a warp each: the waits and issue of
    // both in one took longer than the products.  Small parts are summed first.
    constexpr uint32_t kDescS = (1u << 4) | ((kTok >> 3) << 17) | ((kRows >> 4) << 24);
    constexpr uint32_t kDescO = (1u << 4) | (1u << 16) | ((kHeadDim >> 3) << 17) | ((kRows >> 4) << 24);
    if (warp == kScoreWarp) {
      bool ok = wait(&ctl.q_full, 0, a.fault);
      for (int i = 0; ok && i < ntiles; ++i) {
        const int u = i & 1;
        ok = wait(&ctl.k_full, i & 1, a.fault) && (i < 2 || wait(&ctl.pv_done[u], ((i >> 1) - 1) & 1, a.fault));
        if (!ok) break;
        fence_proxy_async_smem();                 // the other CTAs' stores
        tmem_after_sync();
#pragma unroll
        for (int part = 1; part >= 0; --part)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_f16(tmem + kColS + u * kTok, tmem + kColQ + 8 * k,
                    operand(tiles_k + part * kTile + (k >> 2) * kHalfTile + (k & 3) * 32, 16, 1024), kDescS, part == 0 || k > 0);
        commit<C>(&ctl.s_full[u], false);
        if (i + 1 < ntiles) commit<C>(&ctl.k_empty, true);
      }
    } else {
      for (int i = 0; i < ntiles; ++i) {
        const int u = i & 1;
        if (!wait(&ctl.v_full, i & 1, a.fault) || !wait(&ctl.p_full[u], (i >> 1) & 1, a.fault)) break;
        fence_proxy_async_smem();
        tmem_after_sync();
#pragma unroll
        for (int k = 0; k < kTok / 16; ++k) {
          const uint32_t o = tmem + kColO + u * kHeadDim, p = tmem + kColS + u * kTok + (k >> 1) * 32 + (k & 1) * 8;
          const uint64_t hi = operand(tiles_v + k * 2048, kHalfTile, 1024), lo = operand(tiles_v + kTile + k * 2048, kHalfTile, 1024);
          mma_f16(o, p + 16, hi, kDescO, (i >> 1) % kFlush != 0 || k > 0);
          mma_f16(o, p, lo, kDescO, true);
          mma_f16(o, p, hi, kDescO, true);
        }
        if (i + 1 < ntiles) commit<C>(&ctl.v_empty, true);
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
  const float f_kept = m_kept == m ? 1.f : exp2f(m_kept - m);
  const bool flushed = (ntiles - (st & 1) + 1) / 2 > kFlush;
  auto load_out = [&](int c, float (&x)[32]) {              // 32 dims of this stream's O
    uint32_t o[32];
    tmem_load32(o, out_cols + c);
    tmem_load_wait();
    const float4* kept = kept_row(st & 1, r) + c / 4;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 y = flushed ? __ldcg(kept + j / 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[j] = fmaf(y.x, f_kept, __uint_as_float(o[j]));
      x[j + 1] = fmaf(y.y, f_kept, __uint_as_float(o[j + 1]));
      x[j + 2] = fmaf(y.z, f_kept, __uint_as_float(o[j + 2]));
      x[j + 3] = fmaf(y.w, f_kept, __uint_as_float(o[j + 3]));
    }
  };
  if (joins) {
    ctl.m[st][r] = m;
    ctl.l[st][r] = l;
#pragma unroll 1
    for (int c = 64 * (1 - st); c < 64 * (2 - st); c += 32) {
      float o[32];
      load_out(c, o);
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(rows_out + r * kOutPitch + c + j) =
            have ? make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __syncthreads();
  if (joins) {
    const float m1 = ctl.m[1 - st][r], l1 = ctl.l[1 - st][r];
    const float M = fmaxf(m, m1), ref = M == -INFINITY ? 0.f : M;
    const float back = pow2(-ev), f0 = exp2f(m - ref), f1 = exp2f(m1 - ref);
#pragma unroll 1
    for (int c = 64 * st; c < 64 * (st + 1); c += 32) {
      float o[32];
      load_out(c, o);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        float4* at = reinterpret_cast<float4*>(rows_out + r * kOutPitch + c + j);
        float4 x = *at;
        x = make_float4(x.x * f1, x.y * f1, x.z * f1, x.w * f1);
        if (have) {
          x.x = fmaf(o[j], f0, x.x);
          x.y = fmaf(o[j + 1], f0, x.y);
          x.z = fmaf(o[j + 2], f0, x.z);
          x.w = fmaf(o[j + 3], f0, x.w);
        }
        *at = make_float4(x.x * back, x.y * back, x.z * back, x.w * back);
      }
    }
    if (st == 0 && r < nrows) {
      const size_t at = global_row(r) * n_parts + blockIdx.x;
      if (in_bounds(a.fault, at, n_part_rows(a))) {
        a.part_m[at] = M;
        a.part_l[at] = fmaf(l, f0, l1 * f1);
      }
    }
  }
  tmem_before_sync();
  __syncthreads();
  for (int i = threadIdx.x; i < nrows * 32; i += kThreads) {
    const int rr = i >> 5, c = (i & 31) * 4;
    const size_t at = global_row(rr) * n_parts + blockIdx.x;
    if (in_bounds(a.fault, at, n_part_rows(a)))
      *reinterpret_cast<float4*>(a.part_o + at * kHeadDim + c) = *reinterpret_cast<const float4*>(rows_out + rr * kOutPitch + c);
  }
  if (warp == kScoreWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  cluster_barrier();                              // the other CTAs may still store here until now
}

template <int C, bool kWide, int R>
cudaError_t run(const ServeArgs& a, cudaStream_t stream) {
  static PerDeviceFlag flag;
  using Lay = Layout<C, kWide, R>;
  constexpr uint32_t kMost = kWide ? (Lay::bytes(9) > Lay::bytes(11) ? Lay::bytes(9) : Lay::bytes(11)) : Lay::bytes(R);
  static_assert(kMost <= 227 * 1024 && (!kWide || Lay::bytes(kWideMaxR) <= kMost), "fits an SM");
  static_assert(kOutBytes <= Lay::control(1), "the joined rows fit over tiles and codebooks");
  cudaError_t e = set_smem_limit_once(flag, prefix_mma_kernel<C, kWide, R>, kMost);
  if (e != cudaSuccess) return e;
  e = launch_chained(prefix_book_kernel<C, kWide>, dim3(book_items<C, kWide>(a.R) / kBookThreads, 2 * C, a.n_kv_heads), kBookThreads, a, stream);
  if (e != cudaSuccess) return e;
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
  cfg.dynamicSmemBytes = Lay::bytes(a.R);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, prefix_mma_kernel<C, kWide, R>, a);
}

}  // namespace

cudaError_t launch_prefix_mma(const ServeArgs& a, cudaStream_t stream) {
  if (a.wide) return run<4, true, 0>(a, stream);
  return a.R == 1 ? run<2, false, 1>(a, stream) : run<4, false, 2>(a, stream);
}

}  // namespace cvq
