// C ABI of the serving operators: argument checks on the host, then launches (cvq.h states
// the rules).  As everywhere in the library, nothing is allocated and an argument error is
// returned before any launch.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "serve.cuh"

using namespace cvq;

namespace {

#define CVQ_TRY(expr)                 \
  do {                                \
    const cvq_status st_ = (expr);    \
    if (st_ != CVQ_OK) return st_;    \
  } while (0)

cvq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CVQ_OK : CVQ_ERR_CUDA; }

cvq_status check_ptr(const void* p, unsigned align = 16) {
  if (p == nullptr) return CVQ_ERR_NULL;
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0 ? CVQ_OK : CVQ_ERR_ALIGN;
}

bool is_dtype(int d) { return d == CVQ_F32 || d == CVQ_BF16 || d == CVQ_F16; }
int dtype_bytes(int d) { return d == CVQ_F32 ? 4 : 2; }
bool is_wide(const cvq_shape* s) { return s->group_dim == kWideGroupDim; }
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// CTAs of the tensor-core kernel that share a split (each leaves a partial state)
int prefix_cluster(const cvq_shape* s) { return !is_wide(s) && s->R == 1 ? 2 : 4; }

// Whether the tensor-core kernel takes the call: 16-bit queries, where it is the faster one (both
// hold what fp32 holds).  The other takes 64 rows of a KV head at a time and has less to set up.
// 8 KV heads, R = 1, us in fp32 and here: 1000 tokens of 1, 4, 16, 32 sequences of 4 heads a group
// 11.1 16.1, 11.2 16.4, 17.9 18.7, 33.6 23.2; 2000 tokens of 1, 4, 8, 16 16.4 16.9, 16.9 17.3, 30.6 18.5,
// 31.9 19.5; 192 tokens of 64 21.7 25.3.
bool prefix_on_tensor_cores(const cvq_shape* s, int q_dtype) {
  const int64_t rows = static_cast<int64_t>(s->batch) * (s->n_q_heads / s->n_kv_heads);
  return q_dtype != CVQ_F32 && (s->t_cap >= 2048 || (s->t_cap >= 512 && rows > 64));
}

// partial states of (sequence, query head) rows, 16-byte aligned
size_t parts_bytes(int batch, int n_q_heads, int n_parts) {
  return round16(static_cast<size_t>(batch) * n_q_heads * n_parts * (kHeadDim + 2) * sizeof(float));
}

// What long streams of the tensor-core kernel have summed: two outputs a row and CTA, where a split of a
// full cache has more tiles than two streams sum at once.
size_t kept_bytes(const cvq_shape* s, int n_splits) {
  const int64_t step = kTok * prefix_cluster(s);
  if (((static_cast<int64_t>(s->t_cap) + n_splits - 1) / n_splits + step - 1) / step <= 2 * kFlush) return 0;
  return static_cast<size_t>(s->batch) * s->n_q_heads * n_splits * prefix_cluster(s) * 2 * kHeadDim * sizeof(float);
}

// both codebooks of every KV head
size_t book_bytes(const cvq_shape* s) {
  const size_t entries = is_wide(s) ? kWideGroups * kWideCodes * kWideGroupDim : kGroups * kCodes * kCodeword;
  return 2 * static_cast<size_t>(s->n_kv_heads) * s->R * entries * sizeof(float);
}

void place_parts(ServeArgs& a, void* workspace) {
  const size_t rows = static_cast<size_t>(a.batch) * a.n_q_heads * a.n_parts;
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  a.part_m = a.part_o + rows * kHeadDim;
  a.part_l = a.part_m + rows;
}

cvq_status check_paged(const cvq_paged* p) {
  if (p == nullptr) return CVQ_ERR_NULL;
  if (p->head_dim != kHeadDim) return CVQ_ERR_UNSUPPORTED;
  if (p->kv_dtype != CVQ_BF16 && p->kv_dtype != CVQ_F16) return CVQ_ERR_UNSUPPORTED;
  if (p->batch < 1 || p->n_q_heads < 1 || p->n_kv_heads < 1) return CVQ_ERR_SHAPE;
  if (p->batch > 65535 || p->n_q_heads > 65535) return CVQ_ERR_SHAPE;
  if (p->n_q_heads % p->n_kv_heads != 0) return CVQ_ERR_SHAPE;
  if (p->page_size < 1 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)) != 0) return CVQ_ERR_SHAPE;
  if (p->n_pages < 1 || p->max_pages < 1) return CVQ_ERR_SHAPE;
  if (static_cast<int64_t>(p->max_pages) * p->page_size > INT32_MAX) return CVQ_ERR_SHAPE;
  if (!std::isfinite(p->rope_base) || !(p->rope_base > 1.0f)) return CVQ_ERR_SHAPE;
  const int64_t dense = static_cast<int64_t>(p->n_kv_heads) * p->page_size * kHeadDim;
  if (p->page_stride != 0 && p->page_stride < dense) return CVQ_ERR_SHAPE;
  if (p->page_stride % 8 != 0) return CVQ_ERR_ALIGN;
  // element offsets inside a pool are formed in 64 bits; keep the last one representable
  if ((p->page_stride != 0 ? p->page_stride : dense) > (INT64_MAX / 4) / p->n_pages) return CVQ_ERR_SHAPE;
  const int g = p->n_q_heads / p->n_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8) return CVQ_ERR_UNSUPPORTED;
  return CVQ_OK;
}

int shift_of(int pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

long long stride_of(const cvq_paged* p) {
  return p->page_stride != 0 ? p->page_stride : static_cast<long long>(p->n_kv_heads) * p->page_size * kHeadDim;
}

// a token stride of an append input: whole 16-byte pieces, no shorter than the token's heads
cvq_status check_token_stride(int64_t stride, int heads, int dtype) {
  if (stride < static_cast<int64_t>(heads) * kHeadDim) return CVQ_ERR_SHAPE;
  return stride * dtype_bytes(dtype) % 16 == 0 ? CVQ_OK : CVQ_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t cvq_prefix_workspace_bytes(const cvq_shape* s, int n_splits) {
  if (cvq_partials_bytes(s, n_splits) == 0) return 0;
  // the books' items of 16 bytes leave one peak per 256; two streams a CTA keep an output each
  const int parts = n_splits * prefix_cluster(s);
  return kCounterBytes + parts_bytes(s->batch, s->n_q_heads, parts) + book_bytes(s) + round16(book_bytes(s) / 1024) + kept_bytes(s, n_splits);
}

int cvq_prefix_suggest_splits(const cvq_shape* s, int q_dtype, int sm_count) {
  if (cvq_partials_bytes(s, 1) == 0 || sm_count < 1 || !is_dtype(q_dtype)) return 1;
  const long long rows = static_cast<long long>(s->batch) * (s->n_q_heads / s->n_kv_heads);
  if (prefix_on_tensor_cores(s, q_dtype)) {
    // clusters that fit at once (of 148 SMs 72 pairs, 33 of four), and two steps or more for each
    const int size = prefix_cluster(s);
    const long long units = static_cast<long long>(s->n_kv_heads) * ((rows + 127) / 128);
    const long long fit = size == 2 ? (sm_count - 4) / 2 : sm_count / 4 - 4;
    const long long steps = (static_cast<long long>(s->t_cap) + 64 * size - 1) / (64 * size);
    return static_cast<int>(std::max(1LL, std::min({4096LL, (steps + 1) / 2, fit / units})));
  }
  const long long units = s->n_kv_heads * (rows <= 16 ? 1 : (rows + 63) / 64);
  const long long tiles = std::max(1LL, (static_cast<long long>(s->t_cap) + 63) / 64);
  return static_cast<int>(std::max(1LL, std::min({4096LL, tiles, 2LL * sm_count / units})));
}

cvq_status cvq_prefix_attend(const cvq_shape* s, const void* q, int q_dtype, const float* key_cb,
                             int64_t key_cb_head_stride, const uint8_t* key_codes,
                             const uint8_t* val_codes, const int32_t* prefix_len,
                             const float* val_cb, int64_t val_cb_head_stride, int n_splits,
                             void* workspace, void* out, int out_dtype, float* lse, void* stream) {
  if (s == nullptr) return CVQ_ERR_NULL;
  CVQ_TRY(check_shape_status(s));
  if (!is_dtype(q_dtype) || !is_dtype(out_dtype)) return CVQ_ERR_UNSUPPORTED;
  CVQ_TRY(check_ptr(q));
  CVQ_TRY(check_ptr(key_cb));
  CVQ_TRY(check_ptr(val_cb));
  CVQ_TRY(check_ptr(key_codes));
  CVQ_TRY(check_ptr(val_codes));
  CVQ_TRY(check_ptr(prefix_len, 4));
  CVQ_TRY(check_codebook_stride(s, key_cb_head_stride));
  CVQ_TRY(check_codebook_stride(s, val_cb_head_stride));
  if (n_splits < 1 || n_splits > 4096) return CVQ_ERR_WORKSPACE;
  CVQ_TRY(check_ptr(workspace));
  CVQ_TRY(check_ptr(out));
  CVQ_TRY(check_ptr(lse, 4));
  ServeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q;
  a.q_dtype = q_dtype;
  a.batch = s->batch;
  a.n_q_heads = s->n_q_heads;
  a.n_kv_heads = s->n_kv_heads;
  a.group = s->n_q_heads / s->n_kv_heads;
  const bool tensor = prefix_on_tensor_cores(s, q_dtype);
  a.n_splits = n_splits;
  a.n_parts = tensor ? n_splits * prefix_cluster(s) : n_splits;
  a.lens = prefix_len;
  a.t_cap = s->t_cap;
  a.out = out;
  a.out_dtype = out_dtype;
  a.lse = lse;
  a.key_cb = key_cb;
  a.val_cb = val_cb;
  a.key_cb_stride = key_cb_head_stride;
  a.val_cb_stride = val_cb_head_stride;
  a.key_codes = key_codes;
  a.val_codes = val_codes;
  a.R = s->R;
  a.wide = is_wide(s);
  a.code_bits = s->code_bits == 6 ? 6 : 8;
  phase_turns_host(s->rope_base, &a.phase);
  place_parts(a, workspace);
  char* rest = static_cast<char*>(workspace) + kCounterBytes + parts_bytes(a.batch, a.n_q_heads, a.n_parts);
  a.book = rest;
  a.book_peak = reinterpret_cast<uint32_t*>(rest + book_bytes(s));
  a.kept_o = reinterpret_cast<float*>(rest + book_bytes(s) + round16(book_bytes(s) / 1024));
  if (fault_word_address(&a.fault) != cudaSuccess) return CVQ_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  CVQ_TRY(from_cuda(tensor ? launch_prefix_mma(a, st) : launch_prefix_f32(a, st)));
  return from_cuda(launch_merge(a, st));
}

size_t cvq_paged_workspace_bytes(const cvq_paged* p, int n_splits) {
  if (check_paged(p) != CVQ_OK || n_splits < 1 || n_splits > 4096) return 0;
  return kCounterBytes + parts_bytes(p->batch, p->n_q_heads, n_splits);
}

int cvq_paged_suggest_splits(const cvq_paged* p, int sm_count) {
  if (check_paged(p) != CVQ_OK || sm_count < 1) return 1;
  // For sequences of like lengths.  A split holds 256 tokens or more (512 where there are few splits): on a window of 128 tokens one split takes 7.3 us where
  // two, with their merge, take 14.  Beyond that a CTA per SM carries one sequence best (131071
  // tokens: 18 splits of 8 KV heads 88.9 us, 37 splits 94.8), and of several sequences, whose
  // lengths differ, two CTAs per SM (16 sequences of 1024 to 8192: 3 splits 54.1 us, 2 64.2).
  const long long tokens = static_cast<long long>(p->max_pages) * p->page_size;
  const long long units = static_cast<long long>(p->batch) * p->n_kv_heads;
  const long long ctas = p->batch == 1 ? sm_count : 2LL * sm_count;
  long long n = ctas / units, least = 256;
  if (p->batch > 1 && n < 4) {
    n = (ctas + units - 1) / units;
    least = 512;                                  // 16 sequences of 800: one split 14.1 us, three 19.9
  }
  const long long most = std::max(1LL, tokens / least);
  return static_cast<int>(std::max(1LL, std::min({4096LL, most, n})));
}

cvq_status cvq_paged_append(const cvq_paged* p, int32_t n_tokens, const void* q, int64_t q_stride,
                            const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            int in_dtype, const int32_t* tok_offsets, const int32_t* seq_lens,
                            const int32_t* pos_offsets, const int32_t* page_table, void* k_pages,
                            void* v_pages, void* q_out, void* stream) {
  CVQ_TRY(check_paged(p));
  if (!is_dtype(in_dtype)) return CVQ_ERR_UNSUPPORTED;
  if (n_tokens < 0) return CVQ_ERR_SHAPE;
  if ((q == nullptr) != (q_out == nullptr)) return CVQ_ERR_NULL;
  if (q != nullptr) {
    CVQ_TRY(check_ptr(q));
    CVQ_TRY(check_ptr(q_out));
    CVQ_TRY(check_token_stride(q_stride, p->n_q_heads, in_dtype));
    if (q == q_out && q_stride != static_cast<int64_t>(p->n_q_heads) * kHeadDim) return CVQ_ERR_SHAPE;
  }
  CVQ_TRY(check_ptr(k));
  CVQ_TRY(check_ptr(v));
  CVQ_TRY(check_token_stride(k_stride, p->n_kv_heads, in_dtype));
  CVQ_TRY(check_token_stride(v_stride, p->n_kv_heads, in_dtype));
  CVQ_TRY(check_ptr(tok_offsets, 4));
  CVQ_TRY(check_ptr(seq_lens, 4));
  if (pos_offsets != nullptr) CVQ_TRY(check_ptr(pos_offsets, 4));
  CVQ_TRY(check_ptr(page_table, 4));
  CVQ_TRY(check_ptr(k_pages));
  CVQ_TRY(check_ptr(v_pages));
  if (n_tokens == 0) return CVQ_OK;
  AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.tok_offsets = tok_offsets;
  a.seq_lens = seq_lens;
  a.pos_offsets = pos_offsets;
  a.page_table = page_table;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.q_out = q_out;
  a.n_tokens = n_tokens;
  a.batch = p->batch;
  a.n_q_heads = p->n_q_heads;
  a.n_kv_heads = p->n_kv_heads;
  a.page_shift = shift_of(p->page_size);
  a.n_pages = p->n_pages;
  a.max_pages = p->max_pages;
  a.page_stride = stride_of(p);
  phase_turns_host(p->rope_base, &a.phase);
  if (fault_word_address(&a.fault) != cudaSuccess) return CVQ_ERR_CUDA;
  return from_cuda(launch_paged_append(a, in_dtype, p->kv_dtype, static_cast<cudaStream_t>(stream)));
}

cvq_status cvq_paged_attend(const cvq_paged* p, const void* q, int q_dtype, const void* k_pages,
                            const void* v_pages, const int32_t* page_table,
                            const int32_t* seq_lens, int n_splits, void* workspace,
                            const float* prev_out, const float* prev_lse, void* out, int out_dtype,
                            float* lse, void* stream) {
  CVQ_TRY(check_paged(p));
  if (!is_dtype(q_dtype) || !is_dtype(out_dtype)) return CVQ_ERR_UNSUPPORTED;
  CVQ_TRY(check_ptr(q));
  CVQ_TRY(check_ptr(k_pages));
  CVQ_TRY(check_ptr(v_pages));
  CVQ_TRY(check_ptr(page_table, 4));
  CVQ_TRY(check_ptr(seq_lens, 4));
  if (n_splits < 1 || n_splits > 4096) return CVQ_ERR_WORKSPACE;
  CVQ_TRY(check_ptr(workspace));
  if ((prev_out == nullptr) != (prev_lse == nullptr)) return CVQ_ERR_NULL;
  if (prev_out != nullptr) {
    CVQ_TRY(check_ptr(prev_out));
    CVQ_TRY(check_ptr(prev_lse, 4));
  }
  CVQ_TRY(check_ptr(out));
  CVQ_TRY(check_ptr(lse, 4));
  // in place only where element i of out replaces element i of prev_out
  if (prev_out == out && out_dtype != CVQ_F32) return CVQ_ERR_UNSUPPORTED;
  ServeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q;
  a.q_dtype = q_dtype;
  a.batch = p->batch;
  a.n_q_heads = p->n_q_heads;
  a.n_kv_heads = p->n_kv_heads;
  a.group = p->n_q_heads / p->n_kv_heads;
  a.n_splits = a.n_parts = static_cast<int64_t>(p->batch) * p->n_kv_heads > kCounters ? 1 : n_splits;
  a.t_cap = p->max_pages * p->page_size;
  a.lens = seq_lens;
  a.prev_out = prev_out;
  a.prev_lse = prev_lse;
  a.out = out;
  a.out_dtype = out_dtype;
  a.lse = lse;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.page_table = page_table;
  a.kv_dtype = p->kv_dtype;
  a.page_shift = shift_of(p->page_size);
  a.n_pages = p->n_pages;
  a.max_pages = p->max_pages;
  a.page_stride = stride_of(p);
  place_parts(a, workspace);
  a.counters = static_cast<int*>(workspace);
  if (fault_word_address(&a.fault) != cudaSuccess) return CVQ_ERR_CUDA;
  return from_cuda(launch_paged_attend(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
