// C ABI of cross attention: argument checks, workspaces and launches.
#include <cmath>
#include <utility>

#include "attn_types.h"
#include "op_checks.h"

using namespace ringar;

namespace {

constexpr int kMostDim = 128;
constexpr int64_t kMostPitch = 1 << 24;       // bytes from row to row: the offsets of 128 rows stay below 2^31

// An array of head rows: [batch][rows][heads][dim].
struct Array {
  const char* name;
  const void* p;
  int64_t n[3];            // batch, rows, heads
  int64_t stride[3];
  int64_t dim;
  size_t es;
  bool output;
  size_t align = 16;
};

// First byte after the array (strides have been checked).
unsigned __int128 end_of(const Array& a) {
  unsigned __int128 last = a.dim;
  for (int i = 0; i < 3; i++) last += (unsigned __int128)(a.n[i] - 1) * (uint64_t)a.stride[i];
  return (uintptr_t)a.p + last * a.es;
}

bool empty(const Array& a) { return !a.n[0] || !a.n[1] || !a.n[2]; }

ringar_result_t check_array(Array& a) {
  const std::string name = a.name;
  if (empty(a)) return RINGAR_SUCCESS;
  if (!a.p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + " is null");
  if ((uintptr_t)a.p % a.align)
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + " does not start at a " + std::to_string(a.align) + "-byte boundary");
  for (int i = 0; i < 3; i++) {
    if (a.n[i] == 1) {                         // not used
      a.stride[i] = i == 1 ? a.dim : 0;
      continue;
    }
    if (a.stride[i] < 0) return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + ": a stride below zero");
    if (a.stride[i] > (int64_t)1 << 48) return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + ": a stride beyond 2^48 elements");
    if (a.stride[i] * a.es % 16) return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + ": rows must start at 16-byte boundaries");
  }
  if (a.n[1] > 1 && a.stride[1] * (int64_t)a.es >= kMostPitch) return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + ": row stride of 2^24 bytes or more");
  if (end_of(a) >> 63) return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + " reaches beyond the address space");
  if (!a.output) return RINGAR_SUCCESS;
  // no row of an output over another: from the smallest stride on, each passes all that lies within it
  int by[3] = {0, 1, 2};
  for (int i = 0; i < 3; i++)
    for (int j = i + 1; j < 3; j++)
      if (a.stride[by[j]] < a.stride[by[i]]) std::swap(by[i], by[j]);
  int64_t inner = a.dim;
  for (int i : by) {
    if (a.n[i] == 1) continue;
    if (a.stride[i] < inner) return refuse(RINGAR_ERR_INVALID_ARGUMENT, name + ": rows lie over each other");
    inner = (a.n[i] - 1) * a.stride[i] + inner;
  }
  return RINGAR_SUCCESS;
}

// Every array's own checks, and no output's span over another operand's.
ringar_result_t check_arrays(std::initializer_list<Array*> all) {
  for (Array* a : all) TRY(check_array(*a));
  for (Array* const* o = all.begin(); o != all.end(); o++) {
    if (!(*o)->output || !(*o)->p || empty(**o)) continue;
    for (Array* const* m = all.begin(); m != all.end(); m++) {
      if (m == o || !(*m)->p || empty(**m) || ((*m)->output && m < o)) continue;
      if ((uintptr_t)(*o)->p < end_of(**m) && (uintptr_t)(*m)->p < end_of(**o))
        return refuse(RINGAR_ERR_INVALID_USAGE, std::string((*o)->name) + " overlaps " + (*m)->name);
    }
  }
  return RINGAR_SUCCESS;
}

// A plain vector as an array.
Array vec(const char* name, const void* p, int64_t n, bool output) { return Array{name, p, {p && n ? 1 : 0, 1, 1}, {0, 0, 0}, n, 4, output, 4}; }

template <typename P> ringar_result_t check_sizes(const P* p) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  if (!type_ok(p->dtype)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "attention takes fp16, bf16 or fp32");
  if (!dims_ok({p->batch, p->queries, p->keys, p->heads, p->kv_heads})) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "a size is out of range");
  const int64_t each = 16 / size_of(p->dtype);
  if (p->head_dim < each || p->head_dim > kMostDim || p->head_dim % each)
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "head_dim must be a multiple of " + std::to_string(each) + " up to " + std::to_string(kMostDim));
  if (p->kv_heads == 0 ? p->heads != 0 : p->heads % p->kv_heads != 0)
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "heads must be a multiple of kv_heads");
  if (p->kv_heads && p->queries && p->heads / p->kv_heads > kMaxDim / p->queries)
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "more than 2^31 - 1025 query rows share a key head");
  if ((unsigned __int128)p->batch * p->heads * p->queries >> 48 || (unsigned __int128)p->batch * p->kv_heads * p->keys >> 48)
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "more than 2^48 rows");
  // (the kernels' exponentials are base 2)
  if (!(p->scale > 0.0f) || std::isinf((float)(p->scale * 1.4426950408889634)))
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "scale must be above zero and, times log2(e), finite in fp32");
  return RINGAR_SUCCESS;
}

template <typename P> AttnArgs args_of(const P* p) {
  AttnArgs a = {};
  a.lengths = p->key_lengths;
  a.lse = (float*)p->lse;
  a.batch = (int)p->batch;
  a.queries = (int)p->queries;
  a.keys = (int)p->keys;
  a.heads = (int)p->heads;
  a.kv_heads = (int)p->kv_heads;
  a.dim = (int)p->head_dim;
  a.group = p->kv_heads ? (int)(p->heads / p->kv_heads) : 0;
  a.rows = (int)(a.group * p->queries);
  a.scale = p->scale;
  a.scale2 = (float)(p->scale * 1.4426950408889634);
  return a;
}

HeadRows rows_of(const Array& a) { return HeadRows{a.p, a.stride[0], a.stride[1], a.stride[2]}; }

ringar_result_t check_blocks(const AttnArgs& a) {
  if (attn_blocks(a) > most_blocks(256)) return refuse(RINGAR_ERR_INVALID_USAGE, "more tiles of rows than one launch takes");
  return RINGAR_SUCCESS;
}

}  // namespace

#define ARRAY(field, rows, heads, out) \
  Array{#field, p->field, {p->batch, rows, heads}, {p->field##_strides[0], p->field##_strides[1], p->field##_strides[2]}, p->head_dim, es, out}

static ringar_result_t attention_forward(const ringar_cross_attention_t* p, hipStream_t st) {
  TRY(check_sizes(p));
  const size_t es = size_of(p->dtype);
  Array q = ARRAY(q, p->queries, p->heads, false), k = ARRAY(k, p->keys, p->kv_heads, false), v = ARRAY(v, p->keys, p->kv_heads, false);
  Array y = ARRAY(y, p->queries, p->heads, true);
  Array lengths = vec("key_lengths", p->key_lengths, p->batch, false), lse = vec("lse", p->lse, p->batch * p->heads * p->queries, true);
  TRY(check_arrays({&q, &k, &v, &y, &lengths, &lse}));
  if (empty(q)) return RINGAR_SUCCESS;
  AttnArgs a = args_of(p);
  a.q = rows_of(q);
  a.k = rows_of(k);
  a.v = rows_of(v);
  a.y = rows_of(y);
  plan_attn_forward(p->dtype, a);
  TRY(check_blocks(a));
  Layout l;
  const int64_t parts = a.splits > 1 ? a.splits * p->batch * p->heads * p->queries : 0;
  const size_t at_part = l.add((size_t)parts * a.dim * 4), at_top = l.add((size_t)parts * 8);
  std::lock_guard<std::mutex> lock(g_ws_mu);
  char* ws = nullptr;
  TRY(workspace(st, l.bytes, &ws));
  if (ws) {
    a.part = (float*)(ws + at_part);
    a.part_top = (float*)(ws + at_top);
  }
  HIP_TRY(launch_attn_forward(p->dtype, a, st));
  return RINGAR_SUCCESS;
}

static ringar_result_t attention_backward(const ringar_cross_attention_backward_t* p, hipStream_t st) {
  TRY(check_sizes(p));
  const size_t es = size_of(p->dtype);
  Array dy = ARRAY(dy, p->queries, p->heads, false), y = ARRAY(y, p->queries, p->heads, false);
  Array q = ARRAY(q, p->queries, p->heads, false), k = ARRAY(k, p->keys, p->kv_heads, false), v = ARRAY(v, p->keys, p->kv_heads, false);
  const int64_t d = p->head_dim;
  auto whole = [&](const char* name, void* out, int64_t rows, int64_t heads) {
    return Array{name, out, {out ? p->batch : 0, rows, heads}, {rows * heads * d, heads * d, d}, d, es, true};
  };
  Array dq = whole("dq", p->dq, p->queries, p->heads), dk = whole("dk", p->dk, p->keys, p->kv_heads), dv = whole("dv", p->dv, p->keys, p->kv_heads);
  Array lengths = vec("key_lengths", p->key_lengths, p->batch, false), lse = vec("lse", p->lse, p->batch * p->heads * p->queries, false);
  if (!p->lse && !empty(q)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "lse is null");
  TRY(check_arrays({&dy, &q, &k, &v, &y, &dq, &dk, &dv, &lengths, &lse}));
  const bool want_q = p->dq && !empty(q), want_kv = (p->dk || p->dv) && !empty(k);
  if (!want_q && !want_kv) return RINGAR_SUCCESS;
  AttnArgs a = args_of(p);
  a.q = rows_of(q);
  a.k = rows_of(k);
  a.v = rows_of(v);
  a.y = rows_of(y);
  a.dy = rows_of(dy);
  a.dq = p->dq;
  a.dk = p->dk;
  a.dv = p->dv;
  AttnArgs aq = a, akv = a;
  if (want_q) plan_attn_dq(p->dtype, aq);
  if (want_kv) plan_attn_dkv(p->dtype, akv);
  TRY(check_blocks(aq));
  TRY(check_blocks(akv));
  const int64_t rows = p->batch * p->heads * p->queries, kv_rows = p->batch * p->kv_heads * p->keys;
  Layout l;
  const size_t at_lse2 = l.add((size_t)rows * 4), at_delta = l.add((size_t)rows * 4);
  // the two passes run one after the other and take the same place
  const size_t part_q = want_q && aq.splits > 1 ? (size_t)aq.splits * rows * d * 4 : 0;
  const size_t part_kv = want_kv && akv.splits > 1 ? (size_t)akv.splits * 2 * kv_rows * d * 4 : 0;
  const size_t at_part = l.add(part_q > part_kv ? part_q : part_kv);
  std::lock_guard<std::mutex> lock(g_ws_mu);
  char* ws = nullptr;
  TRY(workspace(st, l.bytes, &ws));
  if (ws) {
    aq.part = akv.part = (float*)(ws + at_part);
    aq.lse2 = akv.lse2 = (float*)(ws + at_lse2);
    aq.delta = akv.delta = (float*)(ws + at_delta);
  }
  if (rows && !want_q) HIP_TRY(launch_attn_delta(p->dtype, aq, st));
  if (want_q) {
    HIP_TRY(launch_attn_dq(p->dtype, aq, st));
    if (aq.splits > 1) HIP_TRY(launch_attn_join(p->dtype, {aq.part, {p->dq, nullptr}, {p->scale, 1.0f}, rows * d, 1, aq.splits}, st));
  }
  if (want_kv) {
    HIP_TRY(launch_attn_dkv(p->dtype, akv, st));
    if (akv.splits > 1) HIP_TRY(launch_attn_join(p->dtype, {akv.part, {p->dk, p->dv}, {p->scale, 1.0f}, kv_rows * d, 2, akv.splits}, st));
  }
  return RINGAR_SUCCESS;
}

extern "C" {

ringar_result_t ringar_cross_attention(const ringar_cross_attention_t* args, ringar_stream_t stream) {
  return guarded([&] { return attention_forward(args, (hipStream_t)stream); });
}

ringar_result_t ringar_cross_attention_backward(const ringar_cross_attention_backward_t* args, ringar_stream_t stream) {
  return guarded([&] { return attention_backward(args, (hipStream_t)stream); });
}

}  // extern "C"
