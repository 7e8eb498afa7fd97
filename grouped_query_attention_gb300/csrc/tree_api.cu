// Entry points of the drafted-token operators (include/gqa.h): argument checks,
// workspace plan, launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/gqa.h"
#include "gqa_host.h"
#include "gqa_internal.h"
#include "host_checks.h"
#include "tree_internal.h"

using gqa::align_up;
using gqa::check_buffers;
using gqa::check_float;
using gqa::check_head_size;
using gqa::check_status_word;
using gqa::cuda_fail;
using gqa::fail;
using gqa::Named;
using gqa::present;
using gqa::shape_is;
using gqa::timed_launch;
using gqa::TreeParams;

namespace {

constexpr long long kElems = 1LL << 40;   // elements of a tensor (byte offsets stay far below 2^63)

// parents: (B, S) or (1, S).
gqa_status check_parents(const gqa_tensor& t, long long B, long long S) {
  if (!present(t) || t.dtype != GQA_I32 || t.ndim != 2 || (t.shape[0] != B && t.shape[0] != 1) || t.shape[1] != S)
    return fail(GQA_ERR_INVALID_ARGUMENT, "parents must be int32 (B or 1, S) = (%lld,%lld)", B, S);
  return GQA_OK;
}

gqa_status check_nodes(long long S) {
  if (S > GQA_MAX_TREE_NODES)
    return fail(GQA_ERR_UNSUPPORTED, "%lld nodes: at most %d", S, GQA_MAX_TREE_NODES);
  return GQA_OK;
}

gqa_status check_ints(const gqa_tensor& t, const char* name, bool optional, int ndim, const int64_t* shape) {
  if (optional && !present(t)) return GQA_OK;
  if (!present(t) || t.dtype != GQA_I32 || !shape_is(t, ndim, shape))
    return fail(GQA_ERR_INVALID_ARGUMENT, "%s must be int32 of shape %s", name, ndim == 1 ? "(B)" : "(B, S)");
  return GQA_OK;
}

struct TreePlan {
  TreeParams P;
  size_t part_o, part_ml, total;   // bytes
};

gqa_status plan_tree(const gqa_handle* h, const gqa_tree_inputs* in, const gqa_tree_outputs* out, TreePlan* pl) {
  if (!h || !in || !out) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL handle, inputs or outputs");
  const gqa_attrs& a = h->attrs;
  if (!a.causal) return fail(GQA_ERR_UNSUPPORTED, "attention of drafted nodes is causal");
  if (a.do_rotary) return fail(GQA_ERR_UNSUPPORTED, "do_rotary does not apply here: rotate with gqa_rotary_axes");
  if (a.k_quant_type != GQA_QUANT_NONE || a.v_quant_type != GQA_QUANT_NONE)
    return fail(GQA_ERR_UNSUPPORTED, "attention of drafted nodes takes float caches");
  if (a.sliding_window_cache) return fail(GQA_ERR_UNSUPPORTED, "sliding_window_cache does not apply to drafted nodes");
  const gqa_tensor& q = in->query;
  gqa_status s;
  if (!present(q)) return fail(GQA_ERR_INVALID_ARGUMENT, "query is required");
  if ((s = check_float(q, "query")) != GQA_OK) return s;
  if (q.ndim != 3 || q.shape[0] < 1 || q.shape[1] < 1 || q.shape[2] < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "query must be a non-empty (B, S, N*H)");
  const long long B = q.shape[0], S = q.shape[1], N = a.num_heads, Nkv = a.kv_num_heads;
  if (q.shape[2] % N) return fail(GQA_ERR_INVALID_ARGUMENT, "query hidden size %lld is not a multiple of num_heads %lld", (long long)q.shape[2], N);
  const long long H = q.shape[2] / N;
  if ((s = check_head_size(H)) != GQA_OK) return s;
  if ((s = check_nodes(S)) != GQA_OK) return s;
  const int64_t kvs[3] = {B, S, Nkv * H};
  for (const gqa_tensor* t : {&in->key, &in->value})
    if (!present(*t) || t->dtype != q.dtype || !shape_is(*t, 3, kvs))
      return fail(GQA_ERR_INVALID_ARGUMENT, "key/value must be (B, S, kv_num_heads*head_size) of the query dtype");
  if ((s = check_parents(in->parents, B, S)) != GQA_OK) return s;
  const int64_t b1[1] = {B}, n1[1] = {N};
  if ((s = check_ints(in->seqlens_k, "seqlens_k", false, 1, b1)) != GQA_OK) return s;
  if ((s = check_ints(in->new_lens, "new_lens", true, 1, b1)) != GQA_OK) return s;
  if (present(in->head_sink) && (in->head_sink.dtype != q.dtype || !shape_is(in->head_sink, 1, n1)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "head_sink must be (num_heads) of the query dtype");
  if (!present(out->output) || out->output.dtype != q.dtype || !shape_is(out->output, 3, q.shape))
    return fail(GQA_ERR_INVALID_ARGUMENT, "output must have the query's shape and dtype");
  const gqa_tensor& c = out->present_key;
  if (!present(c) || c.dtype != q.dtype || c.ndim != 4 || c.shape[0] != B || c.shape[1] != Nkv || c.shape[2] < 1 ||
      c.shape[3] != H || !present(out->present_value) || out->present_value.dtype != q.dtype ||
      !shape_is(out->present_value, 4, c.shape))
    return fail(GQA_ERR_INVALID_ARGUMENT,
                "present_key/value must be (B, kv_num_heads, C, head_size) = (%lld,%lld,C,%lld) of the query dtype", B, Nkv, H);
  const long long C = c.shape[2], T = in->total_sequence_length, G = N / Nkv;
  if (T < 1 || T > C) return fail(GQA_ERR_INVALID_ARGUMENT, "total_sequence_length %lld must be in [1, C = %lld]", T, C);
  if (C > (1LL << 30) || B > 65535 || B * Nkv > 65535 || B * Nkv * C >= (1LL << 31))   // (rows are counted in 32 bits)
    return fail(GQA_ERR_UNSUPPORTED, "present_key/value: tensor too large");
  if (S * N > (1LL << 30) || B * S * N > (1LL << 31) - 65536 || N * H > (1LL << 30)) return fail(GQA_ERR_UNSUPPORTED, "query too large");

  const Named read[] = {{&in->query, "query"}, {&in->key, "key"}, {&in->value, "value"}, {&in->parents, "parents"},
                        {&in->seqlens_k, "seqlens_k"}, {&in->new_lens, "new_lens"}, {&in->head_sink, "head_sink"}};
  const Named written[] = {{&out->output, "output"}, {&out->present_key, "present_key"}, {&out->present_value, "present_value"}};
  if ((s = check_buffers(read, 7, written, 3, nullptr, 0)) != GQA_OK) return s;

  TreeParams& P = pl->P;
  memset(&P, 0, sizeof(P));
  P.B = (int)B; P.S = (int)S; P.N = (int)N; P.Nkv = (int)Nkv; P.G = (int)G; P.H = (int)H;
  P.C = (int)C; P.T = (int)T;
  P.t_type = q.dtype == GQA_F16 ? gqa::kF16 : gqa::kF32;
  // A window that reaches every row hides none; what remains is below 2^30, so the kernels' sums fit 32 bits.
  P.window = a.local_window_size < T ? a.local_window_size : -1;
  P.scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf((float)H);
  P.softcap = gqa::kernel_softcap(a.softcap);
  P.smooth = a.smooth_softmax == 1 ? 1 : 0;
  P.q = q.data; P.k = in->key.data; P.v = in->value.data;
  P.out = out->output.data; P.kc = out->present_key.data; P.vc = out->present_value.data;
  P.seqlens = static_cast<const int*>(in->seqlens_k.data);
  P.new_lens = static_cast<const int*>(in->new_lens.data);
  P.parents = static_cast<const int*>(in->parents.data);
  P.parents_ld = in->parents.shape[0] == B ? (int)S : 0;
  P.sink = in->head_sink.data;
  P.wait_budget = h->wait_budget;
  P.withhold_tile = h->withhold_tile;
  gqa::tree_attn_plan(&P);
  const size_t rows = 2 * ((size_t)P.workers << P.rt_log2);   // two slots a worker
  pl->part_o = align_up(rows * H * sizeof(float));
  pl->part_ml = align_up(rows * 2 * sizeof(float));
  pl->total = pl->part_o + pl->part_ml;
  return GQA_OK;
}

}  // namespace

extern "C" {

gqa_status gqa_tree_workspace_size(const gqa_handle* h, const gqa_tree_inputs* in, const gqa_tree_outputs* out, size_t* bytes) {
  if (!bytes) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL bytes pointer");
  TreePlan pl;
  gqa_status s = plan_tree(h, in, out, &pl);
  if (s != GQA_OK) return s;
  *bytes = pl.total;
  return GQA_OK;
}

gqa_status gqa_tree_describe_plan(const gqa_handle* h, const gqa_tree_inputs* in, const gqa_tree_outputs* out,
                                  gqa_plan_info* info) {
  if (!info) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL info pointer");
  TreePlan pl;
  gqa_status s = plan_tree(h, in, out, &pl);
  if (s != GQA_OK) return s;
  info->regime = pl.P.tc ? GQA_REGIME_PREFILL : GQA_REGIME_DECODE;
  info->launches = 2;
  info->split_len = 1 << pl.P.unit_log2;
  info->max_splits = pl.P.workers;
  info->workspace_bytes = pl.total;
  return GQA_OK;
}

gqa_status gqa_tree_forward(gqa_handle* h, const gqa_tree_inputs* in, const gqa_tree_outputs* out, void* ws, size_t ws_bytes,
                            void* status, void* stream) {
  TreePlan pl;
  gqa_status s = plan_tree(h, in, out, &pl);
  if (s != GQA_OK) return s;
  if ((s = check_status_word(status)) != GQA_OK) return s;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % gqa::kAlign) != 0)
    return fail(GQA_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (ws_bytes < pl.total) return fail(GQA_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, pl.total);
  TreeParams& P = pl.P;
  P.part_o = static_cast<float*>(ws);
  P.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + pl.part_o);
  P.status = static_cast<uint32_t*>(status);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed_launch(h, GQA_KERNEL_TREE_ATTENTION, st, [&] { return gqa::launch_tree_attn(P, st); });
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  e = timed_launch(h, GQA_KERNEL_TREE_MERGE, st, [&] { return gqa::launch_tree_merge(P, st); });
  return e == cudaSuccess ? GQA_OK : cuda_fail(e, "merge launch");
}

gqa_status gqa_tree_verify(gqa_handle* h, const gqa_verify_args* a, void* status, void* stream) {
  if (!h || !a) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL handle or arguments");
  const gqa_tensor& t = a->target_probs;
  gqa_status s;
  if (!present(t)) return fail(GQA_ERR_INVALID_ARGUMENT, "target_probs is required");
  if ((s = check_float(t, "target_probs")) != GQA_OK) return s;
  if (t.ndim != 3 || t.shape[0] < 1 || t.shape[1] < 1 || t.shape[2] < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "target_probs must be a non-empty (B, S, V)");
  const long long B = t.shape[0], S = t.shape[1], V = t.shape[2];
  if ((s = check_nodes(S)) != GQA_OK) return s;
  if (V > (1LL << 30) || B > (1LL << 24) || B * S > kElems / V) return fail(GQA_ERR_UNSUPPORTED, "target_probs: tensor too large");
  if (present(a->draft_probs) && (a->draft_probs.dtype != t.dtype || !shape_is(a->draft_probs, 3, t.shape)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "draft_probs must have target_probs' shape and dtype");
  const int64_t bs[2] = {B, S}, b1[1] = {B};
  if ((s = check_parents(a->parents, B, S)) != GQA_OK) return s;
  if ((s = check_ints(a->tokens, "tokens", false, 2, bs)) != GQA_OK) return s;
  if ((s = check_ints(a->new_lens, "new_lens", true, 1, b1)) != GQA_OK) return s;
  if (!present(a->accept_uniforms) || a->accept_uniforms.dtype != GQA_F32 || !shape_is(a->accept_uniforms, 2, bs))
    return fail(GQA_ERR_INVALID_ARGUMENT, "accept_uniforms must be float32 of shape (B, S)");
  if (!present(a->sample_uniforms) || a->sample_uniforms.dtype != GQA_F32 || !shape_is(a->sample_uniforms, 1, b1))
    return fail(GQA_ERR_INVALID_ARGUMENT, "sample_uniforms must be float32 of shape (B)");
  if ((s = check_ints(a->path, "path", false, 2, bs)) != GQA_OK) return s;
  if ((s = check_ints(a->path_lens, "path_lens", false, 1, b1)) != GQA_OK) return s;
  if ((s = check_ints(a->next_token, "next_token", false, 1, b1)) != GQA_OK) return s;
  if ((s = check_status_word(status)) != GQA_OK) return s;
  const Named read[] = {{&a->tokens, "tokens"}, {&a->parents, "parents"}, {&a->target_probs, "target_probs"},
                        {&a->draft_probs, "draft_probs"}, {&a->accept_uniforms, "accept_uniforms"},
                        {&a->sample_uniforms, "sample_uniforms"}, {&a->new_lens, "new_lens"}};
  const Named written[] = {{&a->path, "path"}, {&a->path_lens, "path_lens"}, {&a->next_token, "next_token"}};
  if ((s = check_buffers(read, 7, written, 3, nullptr, 0)) != GQA_OK) return s;

  gqa::VerifyParams P;
  memset(&P, 0, sizeof(P));
  P.B = (int)B; P.S = (int)S; P.V = V;
  P.half = t.dtype == GQA_F16 ? 1 : 0;
  P.tokens = static_cast<const int*>(a->tokens.data);
  P.parents = static_cast<const int*>(a->parents.data);
  P.parents_ld = a->parents.shape[0] == B ? (int)S : 0;
  P.target = t.data;
  P.draft = a->draft_probs.data;
  P.accept_u = static_cast<const float*>(a->accept_uniforms.data);
  P.sample_u = static_cast<const float*>(a->sample_uniforms.data);
  P.new_lens = static_cast<const int*>(a->new_lens.data);
  P.path = static_cast<int*>(a->path.data);
  P.path_lens = static_cast<int*>(a->path_lens.data);
  P.next = static_cast<int*>(a->next_token.data);
  P.status = static_cast<uint32_t*>(status);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed_launch(h, GQA_KERNEL_TREE_VERIFY, st, [&] { return gqa::launch_tree_verify(P, st); });
  return e == cudaSuccess ? GQA_OK : cuda_fail(e, "verification launch");
}

gqa_status gqa_tree_accept(gqa_handle* h, const gqa_accept_args* a, void* status, void* stream) {
  if (!h || !a || !a->present_keys || !a->present_values) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL handle, arguments or caches");
  if (a->num_layers < 1 || a->num_layers > GQA_MAX_TREE_LAYERS)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_layers must be in [1, %d]", GQA_MAX_TREE_LAYERS);
  const gqa_tensor& c = a->cache;
  gqa_status s;
  if ((s = check_float(c, "cache")) != GQA_OK) return s;
  const long long Nkv = h->attrs.kv_num_heads;
  if (c.ndim != 4 || c.shape[0] < 1 || c.shape[1] != Nkv || c.shape[2] < 1 || c.shape[3] < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "caches must be non-empty (B, kv_num_heads, C, head_size)");
  const long long B = c.shape[0], C = c.shape[2], H = c.shape[3];
  if ((s = check_head_size(H)) != GQA_OK) return s;
  if (C > (1LL << 30) || B > 65535 || B * Nkv > 65535 || B * Nkv * C >= (1LL << 31))
    return fail(GQA_ERR_UNSUPPORTED, "caches: tensor too large");
  if (!present(a->path) || a->path.dtype != GQA_I32 || a->path.ndim != 2 || a->path.shape[0] != B || a->path.shape[1] < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "path must be int32 of shape (B, S)");
  if ((s = check_nodes(a->path.shape[1])) != GQA_OK) return s;
  const int64_t b1[1] = {B};
  if ((s = check_ints(a->path_lens, "path_lens", false, 1, b1)) != GQA_OK) return s;
  if ((s = check_ints(a->seqlens_k, "seqlens_k", false, 1, b1)) != GQA_OK) return s;
  if ((s = check_ints(a->new_lens, "new_lens", true, 1, b1)) != GQA_OK) return s;
  if ((s = check_ints(a->into_seqlens_k, "into_seqlens_k", false, 1, b1)) != GQA_OK) return s;
  if ((s = check_status_word(status)) != GQA_OK) return s;
  const int caches = 2 * a->num_layers;
  gqa::AcceptParams P;
  memset(&P, 0, sizeof(P));
  for (int i = 0; i < caches; ++i) {
    void* data = i & 1 ? a->present_values[i / 2] : a->present_keys[i / 2];
    if (!data || (reinterpret_cast<uintptr_t>(data) & 15u) != 0)
      return fail(GQA_ERR_INVALID_ARGUMENT, "a cache of layer %d is missing or not 16-byte aligned", i / 2);
    P.cache[i] = data;
  }
  // Caches of one size overlap when two of their addresses, in order, are nearer than it; the small tensors one by one.
  const size_t size = gqa::bytes_of(c);
  void* order[2 * gqa::kTreeLayers];
  std::copy(P.cache, P.cache + caches, order);
  std::sort(order, order + caches);
  for (int i = 1; i < caches; ++i)
    if (static_cast<char*>(order[i]) - static_cast<char*>(order[i - 1]) < (ptrdiff_t)size)
      return fail(GQA_ERR_INVALID_ARGUMENT, "a cache overlaps another");
  const Named small[] = {{&a->path, "path"}, {&a->path_lens, "path_lens"}, {&a->seqlens_k, "seqlens_k"}, {&a->new_lens, "new_lens"}};
  const Named into[] = {{&a->into_seqlens_k, "into_seqlens_k"}};
  if ((s = check_buffers(small, 4, into, 1, nullptr, 0)) != GQA_OK) return s;
  for (const Named& n : {small[0], small[1], small[2], small[3], into[0]})
    if (present(*n.t))
      for (int i = 0; i < caches; ++i)
        if (static_cast<char*>(n.t->data) < static_cast<char*>(P.cache[i]) + size &&
            static_cast<char*>(P.cache[i]) < static_cast<char*>(n.t->data) + gqa::bytes_of(*n.t))
          return fail(GQA_ERR_INVALID_ARGUMENT, "a cache overlaps %s", n.name);
  P.B = (int)B; P.S = (int)a->path.shape[1]; P.Nkv = (int)Nkv; P.C = (int)C; P.layers = a->num_layers;
  P.row_bytes = (int)H * (c.dtype == GQA_F16 ? 2 : 4);
  P.path = static_cast<const int*>(a->path.data);
  P.path_lens = static_cast<const int*>(a->path_lens.data);
  P.seqlens = static_cast<const int*>(a->seqlens_k.data);
  P.new_lens = static_cast<const int*>(a->new_lens.data);
  P.into_seqlens = static_cast<int*>(a->into_seqlens_k.data);
  P.status = static_cast<uint32_t*>(status);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed_launch(h, GQA_KERNEL_TREE_ACCEPT, st, [&] { return gqa::launch_tree_accept(P, st); });
  return e == cudaSuccess ? GQA_OK : cuda_fail(e, "row move launch");
}

}  // extern "C"
