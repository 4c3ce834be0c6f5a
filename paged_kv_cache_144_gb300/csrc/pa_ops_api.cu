// pa_ops_api.cu - the extern "C" entry points of the operators around the
// cache (rotary cache write with and without norms, rows read back, attention
// with score modifiers, tree commit, eviction): argument validation and
// dispatch.  No call here allocates device memory.
#include <cmath>
#include <cstring>

#include "../../include/pa.h"
#include "pa_ops.h"

#define PA_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr int kMaxAttendSeqs = 4096;   // the sequences' work sums live in shared memory
constexpr int kMaxGroup = 64;          // query heads per KV head
constexpr int kMaxHeads = 4096;
constexpr int kMaxQueries = 1 << 20;   // per sequence
constexpr int kMaxPath = 256;          // rows a CTA of the commit holds in registers

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool is8bit(int dt) { return dt == PA_FP8_E4M3 || dt == PA_INT8; }
bool cache_dtype(int dt) { return dt == PA_F16 || dt == PA_BF16 || is8bit(dt) || dt == PA_INT4; }
// A tile of a 4-bit cache is whole 16-byte pieces, and its rows a word per 8 values of 128.
bool int4_shape(int head_dim, int block_size) {
  return head_dim == 128 && block_size >= 8 && block_size <= 1024 && (block_size & (block_size - 1)) == 0;
}

// The cache's shape, shared by every call here.
int check_cache(int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int kv_dtype) {
  if (num_kv_heads <= 0 || max_blocks_per_seq <= 0) return PA_ERR_SHAPE;
  if (!cache_dtype(kv_dtype)) return PA_ERR_DTYPE;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_kv_heads > kMaxHeads) return PA_ERR_UNSUPPORTED;
  if (is8bit(kv_dtype) && (head_dim != 128 || num_kv_heads > pa::kMaxHeadParams)) return PA_ERR_UNSUPPORTED;
  if (kv_dtype == PA_INT4 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (block_size < 8 || block_size > 1024 || (block_size & (block_size - 1)) != 0) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size >= (int64_t{1} << 26)) return PA_ERR_SHAPE;
  return PA_OK;
}

int check_pool(const void* k_cache, const void* v_cache, int64_t num_blocks, int num_kv_heads, int block_size) {
  if (!k_cache || !v_cache) return PA_ERR_NULL;
  if (num_blocks <= 0 || num_blocks >= (int64_t{1} << 31) ||
      num_blocks * num_kv_heads * block_size >= (int64_t{1} << 31))
    return PA_ERR_SHAPE;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGN;
  return PA_OK;
}

int shift_of(int block_size) { return __builtin_ctz(static_cast<unsigned>(block_size)); }

int check_attend_shape(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                       int max_blocks_per_seq, int max_q_len, int kv_dtype) {
  if (num_seqs < 0 || num_heads <= 0 || max_q_len <= 0) return PA_ERR_SHAPE;
  const int st = check_cache(num_kv_heads, head_dim, block_size, max_blocks_per_seq, kv_dtype);
  if (st != PA_OK) return st;
  if (num_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
  if (num_heads / num_kv_heads > kMaxGroup || num_heads > kMaxHeads || num_seqs > kMaxAttendSeqs ||
      max_q_len > kMaxQueries)
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Whether the bytes [out, out + out_bytes) meet one of `rows` rows of row_bytes, stride bytes apart from q on.
bool overlaps_rows(const void* out, int64_t out_bytes, const void* q, int64_t rows, int64_t row_bytes, int64_t stride) {
  const int64_t o = static_cast<int64_t>(reinterpret_cast<intptr_t>(out) - reinterpret_cast<intptr_t>(q));
  const int64_t first = o < row_bytes ? 0 : (o - row_bytes) / stride + 1;  // the first row that ends behind out's start
  return first < rows && first * stride < o + out_bytes;
}

}  // namespace

namespace {

// pa_rope_and_cache (norm == nullptr) and pa_norm_rope_and_cache.
int write_rotated(const char* where, const pa_norm_options* norm, void* q_out, int64_t q_out_stride, const void* q,
                  int64_t q_stride, int num_heads, const void* k, const void* v, pa_dtype src_dtype, int64_t k_stride,
                  int64_t v_stride, void* k_cache, void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                  const int64_t* positions, const int64_t* slot_mapping, const float* inv_freq, int rotary_dim,
                  int interleaved, float rope_scale, int num_tokens, int num_kv_heads, int head_dim, int block_size,
                  const float* k_inv_scale, const float* v_inv_scale, const pa_cache_write_options* opt, void* stream) {
  pa_cache_write_options o;
  memset(&o, 0, sizeof(o));
  if (opt) {
    if (opt->struct_size < sizeof(size_t)) return PA_ERR_SHAPE;
    memcpy(&o, opt, opt->struct_size < sizeof(o) ? opt->struct_size : sizeof(o));
  }
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0)
    return PA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_heads > kMaxHeads || num_kv_heads > kMaxHeads) return PA_ERR_UNSUPPORTED;
  if (rotary_dim < (norm ? 0 : 2) || rotary_dim > head_dim || rotary_dim % 2 != 0) return PA_ERR_SHAPE;
  if (norm && !(norm->eps >= 0.f && norm->eps < INFINITY)) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!q_out || !q || !k || !v || !k_cache || !v_cache || !slot_mapping) return PA_ERR_NULL;
  if (rotary_dim > 0 && (!positions || !inv_freq)) return PA_ERR_NULL;
  if (src_dtype != PA_F16 && src_dtype != PA_BF16) return PA_ERR_DTYPE;
  if (kv_dtype != src_dtype && !is8bit(kv_dtype) && kv_dtype != PA_INT4) return PA_ERR_DTYPE;
  if (norm && (norm->q_weight || norm->k_weight) && norm->weight_dtype != PA_F32 && norm->weight_dtype != PA_F16 &&
      norm->weight_dtype != PA_BF16)
    return PA_ERR_DTYPE;
  if (kv_dtype == PA_INT4 && !int4_shape(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  if (is8bit(kv_dtype) && (!k_inv_scale || !v_inv_scale)) return PA_ERR_NULL;
  if (kv_dtype == PA_INT8 && (!o.k_zero_point || !o.v_zero_point)) return PA_ERR_NULL;
  const int64_t qrow = static_cast<int64_t>(num_heads) * head_dim, row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < qrow || q_out_stride < qrow || k_stride < row || v_stride < row) return PA_ERR_SHAPE;
  if (q_out == q && q_out_stride != q_stride) return PA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
      !aligned16(v_cache) || q_stride % 8 != 0 || q_out_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0)
    return PA_ERR_ALIGN;
  if (norm) {
    const uintptr_t most = norm->weight_dtype == PA_F32 ? 3u : 1u;
    if (((reinterpret_cast<uintptr_t>(norm->q_weight) | reinterpret_cast<uintptr_t>(norm->k_weight)) & most) != 0)
      return PA_ERR_ALIGN;
  }
  unsigned int* err = pa::device_error_word();
  if (!err) return PA_ERR_CUDA;
  pa::NormArgs n;
  memset(&n, 0, sizeof(n));
  pa::RopeArgs& a = n.r;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.q = q;
  a.q_stride = q_stride;
  a.num_heads = num_heads;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved;
  a.rope_scale = rope_scale;
  pa::ReshapeArgs& w = a.w;
  w.err = err;
  w.k = k;
  w.v = v;
  w.src_dtype = src_dtype;
  w.k_stride = k_stride;
  w.v_stride = v_stride;
  w.k_cache = k_cache;
  w.v_cache = v_cache;
  w.kv_dtype = kv_dtype;
  w.num_blocks = num_blocks;
  w.slot_mapping = slot_mapping;
  w.num_tokens = num_tokens;
  w.num_kv_heads = num_kv_heads;
  w.head_dim = head_dim;
  w.block_size = block_size;
  w.k_inv_scale = k_inv_scale;
  w.v_inv_scale = v_inv_scale;
  w.k_zero_point = o.k_zero_point;
  w.v_zero_point = o.v_zero_point;
  w.pdl = o.pdl != 0;
  if (!norm && kv_dtype != PA_INT4)
    return pa::cuda_status(pa::launch_rope_and_cache(a, static_cast<cudaStream_t>(stream)), where);
  if (norm) {
    n.q_weight = norm->q_weight;
    n.k_weight = norm->k_weight;
    n.weight_dtype = norm->weight_dtype;
    n.weight_offset = norm->weight_offset;
    n.eps = norm->eps;
  }
  return pa::cuda_status(pa::launch_norm_rope_and_cache(n, static_cast<cudaStream_t>(stream)), where);
}

}  // namespace

PA_EXPORT int pa_rope_and_cache(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, int num_heads,
                                const void* k, const void* v, pa_dtype src_dtype, int64_t k_stride, int64_t v_stride,
                                void* k_cache, void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                                const int64_t* positions, const int64_t* slot_mapping, const float* inv_freq,
                                int rotary_dim, int interleaved, float rope_scale, int num_tokens, int num_kv_heads,
                                int head_dim, int block_size, const float* k_inv_scale, const float* v_inv_scale,
                                const pa_cache_write_options* opt, void* stream) {
  return write_rotated("pa_rope_and_cache launch", nullptr, q_out, q_out_stride, q, q_stride, num_heads, k, v, src_dtype,
                       k_stride, v_stride, k_cache, v_cache, kv_dtype, num_blocks, positions, slot_mapping, inv_freq,
                       rotary_dim, interleaved, rope_scale, num_tokens, num_kv_heads, head_dim, block_size, k_inv_scale,
                       v_inv_scale, opt, stream);
}

PA_EXPORT int pa_norm_rope_and_cache(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, int num_heads,
                                     const void* k, const void* v, pa_dtype src_dtype, int64_t k_stride,
                                     int64_t v_stride, void* k_cache, void* v_cache, pa_dtype kv_dtype,
                                     int64_t num_blocks, const int64_t* positions, const int64_t* slot_mapping,
                                     const float* inv_freq, int rotary_dim, int interleaved, float rope_scale,
                                     int num_tokens, int num_kv_heads, int head_dim, int block_size,
                                     const pa_norm_options* norm, const float* k_inv_scale, const float* v_inv_scale,
                                     const pa_cache_write_options* opt, void* stream) {
  if (!norm) return PA_ERR_NULL;
  if (norm->struct_size < sizeof(size_t)) return PA_ERR_SHAPE;
  pa_norm_options n;
  memset(&n, 0, sizeof(n));
  memcpy(&n, norm, norm->struct_size < sizeof(n) ? norm->struct_size : sizeof(n));
  return write_rotated("pa_norm_rope_and_cache launch", &n, q_out, q_out_stride, q, q_stride, num_heads, k, v, src_dtype,
                       k_stride, v_stride, k_cache, v_cache, kv_dtype, num_blocks, positions, slot_mapping, inv_freq,
                       rotary_dim, interleaved, rope_scale, num_tokens, num_kv_heads, head_dim, block_size, k_inv_scale,
                       v_inv_scale, opt, stream);
}

PA_EXPORT int pa_read_cache(void* k_out, void* v_out, pa_dtype out_dtype, int64_t k_out_stride, int64_t v_out_stride,
                            const void* k_cache, const void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                            const float* k_scale, const float* v_scale, const int64_t* slot_mapping, int num_tokens,
                            int num_kv_heads, int head_dim, int block_size, const pa_cache_write_options* opt,
                            void* stream) {
  pa_cache_write_options o;
  memset(&o, 0, sizeof(o));
  if (opt) {
    if (opt->struct_size < sizeof(size_t)) return PA_ERR_SHAPE;
    memcpy(&o, opt, opt->struct_size < sizeof(o) ? opt->struct_size : sizeof(o));
  }
  if (num_tokens < 0 || num_kv_heads <= 0) return PA_ERR_SHAPE;
  if (!cache_dtype(kv_dtype)) return PA_ERR_DTYPE;
  // (8-bit rows of 64 too: the writes make them)
  if ((head_dim != 64 && head_dim != 128) || num_kv_heads > kMaxHeads) return PA_ERR_UNSUPPORTED;
  if (kv_dtype == PA_INT4 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (block_size < 8 || block_size > 1024 || (block_size & (block_size - 1)) != 0) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!k_out || !v_out || !slot_mapping) return PA_ERR_NULL;
  if (out_dtype != PA_F32 && out_dtype != PA_F16 && out_dtype != PA_BF16) return PA_ERR_DTYPE;
  if (is8bit(kv_dtype) && (!k_scale || !v_scale)) return PA_ERR_NULL;
  if (kv_dtype == PA_INT8 && (!o.k_zero_point || !o.v_zero_point)) return PA_ERR_NULL;
  const int ps = check_pool(k_cache, v_cache, num_blocks, num_kv_heads, block_size);
  if (ps != PA_OK) return ps;
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (k_out_stride < row || v_out_stride < row) return PA_ERR_SHAPE;
  if (num_tokens * static_cast<int64_t>(num_kv_heads) >= (int64_t{1} << 35)) return PA_ERR_SHAPE;  // CTAs of 32 rows
  const int64_t piece = out_dtype == PA_F32 ? 4 : 8;  // elements of 16 bytes
  if (!aligned16(k_out) || !aligned16(v_out) || k_out_stride % piece != 0 || v_out_stride % piece != 0) return PA_ERR_ALIGN;
  const int64_t bytes = out_dtype == PA_F32 ? 4 : 2;
  if (k_out == v_out ||
      overlaps_rows(k_out, ((num_tokens - 1) * k_out_stride + row) * bytes, v_out, num_tokens, row * bytes,
                    v_out_stride * bytes)) {
    // (rows of one buffer may alternate: K and V side by side in each token's row)
    const int64_t apart = static_cast<int64_t>(reinterpret_cast<intptr_t>(v_out) - reinterpret_cast<intptr_t>(k_out));
    const int64_t stride = k_out_stride * bytes, at = ((apart % stride) + stride) % stride;
    if (k_out_stride != v_out_stride || at < row * bytes || at + row * bytes > stride) return PA_ERR_SHAPE;
  }
  pa::ReadArgs a;
  memset(&a, 0, sizeof(a));
  a.err = pa::device_error_word();
  if (!a.err) return PA_ERR_CUDA;
  a.k_out = k_out;
  a.v_out = v_out;
  a.out_dtype = out_dtype;
  a.k_stride = k_out_stride;
  a.v_stride = v_out_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.kv_dtype = kv_dtype;
  a.num_blocks = num_blocks;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_zero_point = o.k_zero_point;
  a.v_zero_point = o.v_zero_point;
  a.slots = slot_mapping;
  a.num_tokens = num_tokens;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.block_shift = shift_of(block_size);
  a.pdl = o.pdl != 0;
  return pa::cuda_status(pa::launch_read_cache(a, static_cast<cudaStream_t>(stream)), "pa_read_cache launch");
}

PA_EXPORT size_t pa_attend_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                           int block_size, int max_blocks_per_seq, int max_q_len, pa_dtype kv_dtype,
                                           int accumulate) {
  if (check_attend_shape(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, max_q_len,
                         kv_dtype) != PA_OK ||
      (accumulate && max_q_len != 1))
    return static_cast<size_t>(-1);
  return pa::attend_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                                    max_q_len, kv_dtype, accumulate != 0);
}

PA_EXPORT int pa_attend(void* out, pa_dtype out_dtype, const void* q, pa_dtype q_dtype, int64_t q_stride,
                        const void* k_cache, const void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                        const float* k_scale, const float* v_scale, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_starts, int max_q_len,
                        int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim, float scale,
                        int block_size, void* workspace, size_t workspace_bytes, const pa_attend_options* opt,
                        void* stream) {
  pa_attend_options o;
  memset(&o, 0, sizeof(o));
  if (opt) {
    if (opt->struct_size < sizeof(size_t)) return PA_ERR_SHAPE;
    memcpy(&o, opt, opt->struct_size < sizeof(o) ? opt->struct_size : sizeof(o));
  }
  const int sh = check_attend_shape(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                                    max_q_len, kv_dtype);
  if (sh != PA_OK) return sh;
  if (num_tokens < 0 || !(o.softcap >= 0.f) || std::isinf(o.softcap) || o.window < 0) return PA_ERR_SHAPE;
  // outside these the score's float32 form loses too much: its error is about 2^-21 softcap
  if (o.softcap > 0.f && (o.softcap < 0x1p-10f || o.softcap > 512.f)) return PA_ERR_UNSUPPORTED;
  if (o.window > 0 && (o.prefix_lens || o.tree_mask)) return PA_ERR_UNSUPPORTED;
  if (o.sinks < 0) return PA_ERR_SHAPE;
  if (o.sinks > 0 && (o.prefix_lens || o.tree_mask)) return PA_ERR_UNSUPPORTED;
  if (o.tree_mask && (o.slopes || o.prefix_lens)) return PA_ERR_UNSUPPORTED;
  if (o.tree_mask && (o.tree_words <= 0 || static_cast<int64_t>(o.tree_words) * 64 < max_q_len)) return PA_ERR_SHAPE;
  if (o.mass && max_q_len != 1) return PA_ERR_UNSUPPORTED;
  const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  if (o.mass && (o.mass_stride_head < cap || o.mass_stride_seq < o.mass_stride_head * num_kv_heads))
    return PA_ERR_SHAPE;
  if (num_seqs == 0) return PA_OK;
  if (!q_starts && (max_q_len != 1 || num_tokens < num_seqs)) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!out || !q || !block_tables || !seq_lens) return PA_ERR_NULL;
  if (out_dtype != PA_F32 && out_dtype != PA_F16 && out_dtype != PA_BF16) return PA_ERR_DTYPE;
  if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_ERR_DTYPE;
  if (kv_dtype != q_dtype && !is8bit(kv_dtype) && kv_dtype != PA_INT4) return PA_ERR_DTYPE;
  if (is8bit(kv_dtype) && (!k_scale || !v_scale)) return PA_ERR_NULL;
  if (kv_dtype == PA_INT8 && (!o.k_zero_point || !o.v_zero_point)) return PA_ERR_NULL;
  const int ps = check_pool(k_cache, v_cache, num_blocks, num_kv_heads, block_size);
  if (ps != PA_OK) return ps;
  if (q_stride < static_cast<int64_t>(num_heads) * head_dim) return PA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out) || q_stride % 8 != 0) return PA_ERR_ALIGN;
  // the work of a call is counted in tiles of 128 positions per row tile, or in units of 32 positions, in 32 bits
  if ((static_cast<int64_t>(num_tokens) * (num_heads / num_kv_heads) / 128 + num_seqs) * num_kv_heads * (cap / 128 + 2) >=
      (int64_t{1} << 31))
    return PA_ERR_SHAPE;
  if (static_cast<int64_t>(num_seqs) * num_kv_heads * (cap / 32 + 4) >= (int64_t{1} << 31)) return PA_ERR_SHAPE;
  const int64_t row = static_cast<int64_t>(num_heads) * head_dim;
  if (overlaps_rows(out, num_tokens * row * (out_dtype == PA_F32 ? 4 : 2), q, num_tokens, row * 2, q_stride * 2))
    return PA_ERR_SHAPE;
  unsigned int* err = pa::device_error_word();
  if (!err) return PA_ERR_CUDA;
  pa::AttendParams p;
  memset(&p, 0, sizeof(p));
  p.out = out;
  p.out_dtype = out_dtype;
  p.q = q;
  p.q_dtype = q_dtype;
  p.q_stride = q_stride;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_dtype = kv_dtype;
  p.num_blocks = num_blocks;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_zero_point = o.k_zero_point;
  p.v_zero_point = o.v_zero_point;
  p.block_tables = block_tables;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.seq_lens = seq_lens;
  p.q_starts = q_starts;
  p.max_q_len = max_q_len;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.head_dim = head_dim;
  p.scale = scale;
  p.block_size = block_size;
  p.block_shift = shift_of(block_size);
  p.softcap = o.softcap;
  p.slopes = o.slopes;
  p.window = o.window;
  p.sinks = o.window > 0 ? (o.sinks < cap ? o.sinks : static_cast<int>(cap)) : 0;  // (without a window everything is seen)
  p.prefix_lens = o.prefix_lens;
  p.tree_mask = o.tree_mask;
  p.tree_words = o.tree_words;
  p.mass = o.mass;
  p.mass_stride_seq = o.mass_stride_seq;
  p.mass_stride_head = o.mass_stride_head;
  p.err = err;
  p.pdl = o.pdl != 0;
  p.wait_limit_ns = pa::wait_limit_ns();
  return pa::launch_attend(p, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

PA_EXPORT int pa_commit_tree(void* k_cache, void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                             const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                             const int32_t* q_starts, const int32_t* path, const int32_t* path_lens, int max_path,
                             int32_t* new_lens, int num_seqs, int num_kv_heads, int head_dim, int block_size,
                             void* stream) {
  const int sh = check_cache(num_kv_heads, head_dim, block_size, max_blocks_per_seq, kv_dtype);
  if (sh != PA_OK) return sh;
  if (kv_dtype == PA_INT4) return PA_ERR_UNSUPPORTED;
  if (num_seqs < 0 || max_path < 1) return PA_ERR_SHAPE;
  if (max_path > kMaxPath || num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!block_tables || !seq_lens || !q_starts || !path || !path_lens || !new_lens) return PA_ERR_NULL;
  if (new_lens == seq_lens) return PA_ERR_SHAPE;
  const int ps = check_pool(k_cache, v_cache, num_blocks, num_kv_heads, block_size);
  if (ps != PA_OK) return ps;
  pa::CommitArgs a;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_blocks = num_blocks;
  a.row_bytes = head_dim * (is8bit(kv_dtype) ? 1 : 2);
  a.block_tables = block_tables;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.seq_lens = seq_lens;
  a.q_starts = q_starts;
  a.path = path;
  a.path_lens = path_lens;
  a.max_path = max_path;
  a.new_lens = new_lens;
  a.num_seqs = num_seqs;
  a.num_kv_heads = num_kv_heads;
  a.block_size = block_size;
  a.block_shift = shift_of(block_size);
  a.err = pa::device_error_word();
  if (!a.err) return PA_ERR_CUDA;
  return pa::cuda_status(pa::launch_commit_tree(a, static_cast<cudaStream_t>(stream)), "pa_commit_tree launch");
}

PA_EXPORT int pa_evict(void* k_cache, void* v_cache, pa_dtype kv_dtype, int64_t num_blocks, const float* mass,
                       int64_t mass_stride_seq, int64_t mass_stride_head, const int32_t* block_tables,
                       int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* dst_tables, int max_dst_blocks,
                       int32_t* kept, float* mass_out, int32_t* new_lens, int num_seqs, int num_kv_heads,
                       int head_dim, int block_size, int budget, int recent, int sinks, void* stream) {
  const int sh = check_cache(num_kv_heads, head_dim, block_size, max_blocks_per_seq, kv_dtype);
  if (sh != PA_OK) return sh;
  if (kv_dtype == PA_INT4) return PA_ERR_UNSUPPORTED;
  const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  if (num_seqs < 0 || budget < 1 || budget >= (1 << 26) || recent < 0 || sinks < 0 || max_dst_blocks < 1 ||
      static_cast<int64_t>(recent) + sinks > budget)
    return PA_ERR_SHAPE;
  if (static_cast<int64_t>(max_dst_blocks) * block_size < (budget < cap ? budget : cap)) return PA_ERR_SHAPE;
  if (mass_stride_head < cap || mass_stride_seq < mass_stride_head * num_kv_heads) return PA_ERR_SHAPE;
  if (num_seqs > 65535 || num_kv_heads > 32767) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!mass || !block_tables || !seq_lens || !dst_tables || !kept || !mass_out || !new_lens) return PA_ERR_NULL;
  if (new_lens == seq_lens || mass_out == mass) return PA_ERR_SHAPE;
  const int ps = check_pool(k_cache, v_cache, num_blocks, num_kv_heads, block_size);
  if (ps != PA_OK) return ps;
  pa::EvictArgs a;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_blocks = num_blocks;
  a.row_bytes = head_dim * (is8bit(kv_dtype) ? 1 : 2);
  a.mass = mass;
  a.mass_stride_seq = mass_stride_seq;
  a.mass_stride_head = mass_stride_head;
  a.block_tables = block_tables;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.seq_lens = seq_lens;
  a.dst_tables = dst_tables;
  a.max_dst_blocks = max_dst_blocks;
  a.kept = kept;
  a.mass_out = mass_out;
  a.new_lens = new_lens;
  a.num_seqs = num_seqs;
  a.num_kv_heads = num_kv_heads;
  a.block_size = block_size;
  a.block_shift = shift_of(block_size);
  a.budget = budget;
  a.recent = recent;
  a.sinks = sinks;
  a.err = pa::device_error_word();
  if (!a.err) return PA_ERR_CUDA;
  return pa::cuda_status(pa::launch_evict(a, static_cast<cudaStream_t>(stream)), "pa_evict launch");
}
