// libbfp8 C ABI, second part: argument validation and dispatch of the entry
// points of include/bfp8_attention.h.  As in api.cpp, every argument is
// checked on the host before the first HIP call.

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "attention.h"

using namespace bfp8;

namespace {

constexpr int64_t kMaxRow = int64_t(1) << 22;   // elements; see head_rows
constexpr int64_t kMaxHead = int64_t(1) << 40;  // elements
constexpr int64_t kMaxTile = 512;  // rows or keys of a tile and the next at most
constexpr int kClearAll =
    BFP8_CLEAR_O | BFP8_CLEAR_LSE | BFP8_CLEAR_DQ | BFP8_CLEAR_DK | BFP8_CLEAR_DV;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A tensor of heads whose values have `size` bytes.
bfp8_status check_heads(const void* data, int64_t row, int64_t head, int64_t size, int64_t heads,
                        int64_t dim) {
  if (data == nullptr) return BFP8_ERR_NULL;
  if (!aligned16(data)) return BFP8_ERR_ALIGN;
  if (row < dim || row > kMaxRow || head < 0 || head > kMaxHead) return BFP8_ERR_SHAPE;
  if (heads > 1 && head < dim) return BFP8_ERR_SHAPE;
  if (row * size % 16 != 0 || (heads > 1 && head * size % 16 != 0)) return BFP8_ERR_ALIGN;
  return BFP8_OK;
}

bfp8_status check_shape(const bfp8_attention_shape* s) {
  if (s == nullptr) return BFP8_ERR_NULL;
  const int64_t limit = int64_t(1) << 31;
  if (s->batch < 0 || s->total_q < 0 || s->total_k < 0 || s->batch >= limit ||
      s->total_q >= limit || s->total_k >= limit)
    return BFP8_ERR_SHAPE;
  // a query's place and a key's, and a tile past either, are added in 32 bits
  if (s->total_q + s->total_k > limit - kMaxTile) return BFP8_ERR_SHAPE;
  if (s->heads <= 0 || s->kv_heads <= 0 || s->heads % s->kv_heads != 0) return BFP8_ERR_SHAPE;
  // rows of a kv head (queries times heads of its group) are counted in 32 bits
  if (s->total_q * (s->heads / s->kv_heads) >= limit) return BFP8_ERR_SHAPE;
  if (s->head_dim <= 0 || s->head_dim > 128 || s->head_dim % 8 != 0) return BFP8_ERR_SHAPE;
  if ((s->causal & ~(1 | kClearAll)) != 0) return BFP8_ERR_SHAPE;
  if (!(s->scale > 0.0f) || isinf(s->scale)) return BFP8_ERR_SHAPE;
  if (s->batch == 0) return s->total_q == 0 && s->total_k == 0 ? BFP8_OK : BFP8_ERR_SHAPE;
  if (s->cu_q == nullptr && s->total_q % s->batch != 0) return BFP8_ERR_SHAPE;
  if (s->cu_k == nullptr && s->total_k % s->batch != 0) return BFP8_ERR_SHAPE;
  return BFP8_OK;
}

AttentionArgs make_args(const bfp8_attention_shape& s) {
  AttentionArgs a{};
  a.cu_q = s.cu_q;
  a.cu_k = s.cu_k;
  a.k_lens = s.k_lens;
  a.batch = static_cast<int>(s.batch);
  a.total_q = static_cast<int>(s.total_q);
  a.total_k = static_cast<int>(s.total_k);
  a.heads = s.heads;
  a.kv_heads = s.kv_heads;
  a.group = s.heads / s.kv_heads;
  a.head_dim = s.head_dim;
  a.causal = s.causal & 1;
  a.scale = s.scale;
  a.scale_log2 = static_cast<float>(s.scale * 1.4426950408889634);
  return a;
}

template <typename H>
Heads as_heads(const H& t) {
  return Heads{static_cast<uint16_t*>(const_cast<void*>(static_cast<const void*>(t.data))), t.row,
               t.head};
}

// The checks of a query-side (rows = total_q) or key-side tensor, which may be
// NULL where it has no rows.
template <typename H>
bfp8_status check_tensor(const H& t, int64_t rows, int heads, int dim) {
  return rows == 0 ? BFP8_OK : check_heads(t.data, t.row, t.head, 2, heads, dim);
}

bfp8_status scan_heads(const bfp8_heads& t, int64_t rows, int heads, int dim, hipStream_t stream) {
  if (rows == 0) return BFP8_OK;
  if (t.head == dim) return check_finite(t.data, BFP8_IN_BF16, rows, (int64_t)heads * dim, t.row, stream);
  for (int h = 0; h < heads; ++h) {
    const bfp8_status st = check_finite(static_cast<const uint16_t*>(t.data) + h * t.head,
                                        BFP8_IN_BF16, rows, dim, t.row, stream);
    if (st != BFP8_OK) return st;
  }
  return BFP8_OK;
}

// Debug mode: q whole, k and v where every row is used (rows past a sequence's
// used length may hold anything).
bfp8_status scan_inputs(const bfp8_attention_shape& s, const bfp8_heads& q, const bfp8_heads& k,
                        const bfp8_heads& v, hipStream_t stream) {
  bfp8_status st = scan_heads(q, s.total_q, s.heads, s.head_dim, stream);
  if (st != BFP8_OK || s.k_lens != nullptr) return st;
  st = scan_heads(k, s.total_k, s.kv_heads, s.head_dim, stream);
  return st != BFP8_OK ? st : scan_heads(v, s.total_k, s.kv_heads, s.head_dim, stream);
}

}  // namespace

extern "C" {

bfp8_status bfp8_rope_table(float* table, int64_t positions, int rot_dim, double base,
                            bfp8_rope_scaling scaling, double factor, int64_t original_length,
                            hipStream_t stream) {
  if (scaling < BFP8_ROPE_NONE || scaling > BFP8_ROPE_YARN) return BFP8_ERR_LAYOUT;
  if (positions < 0 || rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > 512) return BFP8_ERR_SHAPE;
  if (positions >= (int64_t(1) << 31)) return BFP8_ERR_SHAPE;
  if (!(base > 0.0) || isinf(base)) return BFP8_ERR_SHAPE;
  if (scaling != BFP8_ROPE_NONE && (!(factor >= 1.0) || isinf(factor))) return BFP8_ERR_SHAPE;
  if (scaling == BFP8_ROPE_YARN && original_length <= 0) return BFP8_ERR_SHAPE;
  if (positions == 0) return BFP8_OK;
  if (table == nullptr) return BFP8_ERR_NULL;
  if (!aligned16(table)) return BFP8_ERR_ALIGN;
  return launch_rope_table(table, positions, rot_dim, base, factor,
                           static_cast<double>(original_length), scaling, stream);
}

bfp8_status bfp8_rope(const void* x, int64_t x_row, int64_t x_head, void* y, int64_t y_row,
                      int64_t y_head, bfp8_in_dtype dt, int64_t tokens, int64_t heads,
                      int head_dim, int rot_dim, bfp8_rope_layout layout, const float* table,
                      int64_t table_rows, const int32_t* positions, int inverse,
                      hipStream_t stream) {
  if (dt != BFP8_IN_BF16 && dt != BFP8_IN_F32) return BFP8_ERR_DTYPE;
  if (layout != BFP8_ROPE_HALF && layout != BFP8_ROPE_INTERLEAVED) return BFP8_ERR_LAYOUT;
  const int64_t size = dt == BFP8_IN_F32 ? 4 : 2;
  if (tokens < 0 || heads < 0 || table_rows < 0) return BFP8_ERR_SHAPE;
  if (head_dim <= 0 || head_dim > 512 || head_dim * size % 16 != 0) return BFP8_ERR_SHAPE;
  if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 2 != 0) return BFP8_ERR_SHAPE;
  if (inverse != 0 && inverse != 1) return BFP8_ERR_SHAPE;
  if (tokens == 0 || heads == 0) return BFP8_OK;
  if (tokens >= (int64_t(1) << 31) || heads >= (int64_t(1) << 31) ||
      tokens * heads >= (int64_t(1) << 31))
    return BFP8_ERR_SHAPE;
  bfp8_status st = check_heads(x, x_row, x_head, size, heads, head_dim);
  if (st == BFP8_OK) st = check_heads(y, y_row, y_head, size, heads, head_dim);
  if (st != BFP8_OK) return st;
  if (x == y && (x_row != y_row || (heads > 1 && x_head != y_head))) return BFP8_ERR_SHAPE;
  // without rows in the table every position is outside it
  if (table_rows > 0 && table == nullptr) return BFP8_ERR_NULL;
  if (table_rows == 0) return BFP8_ERR_SHAPE;
  if (!aligned16(table)) return BFP8_ERR_ALIGN;
  RopeArgs a{x,     y,     x_row,    x_head,  y_row, y_head,     tokens,
             heads, head_dim, rot_dim, table, table_rows, positions, inverse};
  return launch_rope(a, dt, layout == BFP8_ROPE_INTERLEAVED, stream);
}

size_t bfp8_attention_workspace_bytes(const bfp8_attention_shape* shape, int backward) {
  if (check_shape(shape) != BFP8_OK || (backward != 0 && backward != 1))
    return static_cast<size_t>(-1);
  const AttentionArgs a = make_args(*shape);
  return backward ? attention_backward_workspace(a) : attention_forward_workspace(a);
}

bfp8_status bfp8_attention_forward(const bfp8_attention_shape* shape, bfp8_heads q, bfp8_heads k,
                                   bfp8_heads v, bfp8_heads_out o, float* lse, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  bfp8_status st = check_shape(shape);
  if (st != BFP8_OK) return st;
  const bfp8_attention_shape& s = *shape;
  if (s.total_q == 0) return BFP8_OK;
  if ((st = check_tensor(q, s.total_q, s.heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(k, s.total_k, s.kv_heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(v, s.total_k, s.kv_heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(o, s.total_q, s.heads, s.head_dim)) != BFP8_OK) return st;
  if (lse == nullptr) return BFP8_ERR_NULL;
  if (!aligned16(lse) || (workspace != nullptr && !aligned16(workspace))) return BFP8_ERR_ALIGN;
  if (debug_checks_enabled() && (st = scan_inputs(s, q, k, v, stream)) != BFP8_OK) return st;
  AttentionArgs a = make_args(s);
  a.q = as_heads(q);
  a.k = as_heads(k);
  a.v = as_heads(v);
  a.o = as_heads(o);
  a.lse = lse;
  if (s.cu_q != nullptr) a.clear = s.causal & (BFP8_CLEAR_O | BFP8_CLEAR_LSE);
  return launch_attention_forward(a, workspace, workspace_bytes, stream);
}

bfp8_status bfp8_attention_backward(const bfp8_attention_shape* shape, bfp8_heads q, bfp8_heads k,
                                    bfp8_heads v, bfp8_heads o, const float* lse, bfp8_heads dout,
                                    bfp8_heads_out dq, bfp8_heads_out dk, bfp8_heads_out dv,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  bfp8_status st = check_shape(shape);
  if (st != BFP8_OK) return st;
  const bfp8_attention_shape& s = *shape;
  if (s.total_q == 0 && s.total_k == 0) return BFP8_OK;
  if ((st = check_tensor(q, s.total_q, s.heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(k, s.total_k, s.kv_heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(v, s.total_k, s.kv_heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(o, s.total_q, s.heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(dout, s.total_q, s.heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(dq, s.total_q, s.heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(dk, s.total_k, s.kv_heads, s.head_dim)) != BFP8_OK) return st;
  if ((st = check_tensor(dv, s.total_k, s.kv_heads, s.head_dim)) != BFP8_OK) return st;
  if (s.total_q > 0 && lse == nullptr) return BFP8_ERR_NULL;
  if (!aligned16(lse) || !aligned16(workspace)) return BFP8_ERR_ALIGN;
  const size_t need = bfp8_attention_workspace_bytes(shape, 1);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BFP8_ERR_WORKSPACE;
  if (debug_checks_enabled()) {
    if ((st = scan_inputs(s, q, k, v, stream)) != BFP8_OK) return st;
    if ((st = scan_heads(dout, s.total_q, s.heads, s.head_dim, stream)) != BFP8_OK) return st;
  }
  AttentionArgs a = make_args(s);
  a.q = as_heads(q);
  a.k = as_heads(k);
  a.v = as_heads(v);
  a.o = as_heads(o);
  a.dout = as_heads(dout);
  a.dq = as_heads(dq);
  a.dk = as_heads(dk);
  a.dv = as_heads(dv);
  a.lse = const_cast<float*>(lse);
  if (s.cu_q != nullptr) a.clear |= s.causal & BFP8_CLEAR_DQ;
  if (s.cu_k != nullptr) a.clear |= s.causal & (BFP8_CLEAR_DK | BFP8_CLEAR_DV);
  return launch_attention_backward(a, workspace, stream);
}

}  // extern "C"
