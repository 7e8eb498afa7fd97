// Entry points of the multi-axis rotary, the block-scaled int8 cache and its
// eviction (include/gqa.h): argument checks, workspace plan, launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/gqa.h"
#include "block_internal.h"
#include "gqa_host.h"
#include "gqa_internal.h"

using gqa::align_up;
using gqa::BlockParams;
using gqa::cuda_fail;
using gqa::fail;
using gqa::present;
using gqa::shape_is;
using gqa::timed_launch;

namespace {

size_t dtype_size(int32_t d) {
  switch (d) {
    case GQA_F32:
    case GQA_I32: return 4;
    case GQA_F16:
    case GQA_BF16: return 2;
    case GQA_I8:
    case GQA_U8: return 1;
  }
  return 0;
}

size_t bytes_of(const gqa_tensor& t) {
  size_t n = dtype_size(t.dtype);
  for (int i = 0; i < t.ndim; ++i) n *= (size_t)t.shape[i];
  return n;
}

bool overlap(const gqa_tensor& a, const gqa_tensor& b) {
  if (!present(a) || !present(b)) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.data), pb = reinterpret_cast<uintptr_t>(b.data);
  return pa < pb + bytes_of(b) && pb < pa + bytes_of(a);
}

struct Named {
  const gqa_tensor* t;
  const char* name;
};

// Alignment of every tensor, and that no written one overlaps another (`same`
// pairs may be one buffer).
gqa_status check_buffers(const Named* read, int nread, const Named* written, int nwritten, const gqa_tensor* same[][2],
                         int nsame) {
  for (int k = 0; k < nread + nwritten; ++k) {
    const Named& n = k < nread ? read[k] : written[k - nread];
    gqa_status s = gqa::check_aligned(*n.t, n.name);
    if (s != GQA_OK) return s;
  }
  for (int i = 0; i < nwritten; ++i) {
    for (int k = 0; k < nread + i; ++k) {
      const Named& n = k < nread ? read[k] : written[k - nread];
      if (!overlap(*written[i].t, *n.t)) continue;
      bool ok = false;
      for (int x = 0; x < nsame; ++x)
        ok |= same[x][0] == written[i].t && same[x][1] == n.t && written[i].t->data == n.t->data;
      if (!ok) return fail(GQA_ERR_INVALID_ARGUMENT, "%s overlaps %s", written[i].name, n.name);
    }
  }
  return GQA_OK;
}

gqa_status check_float(const gqa_tensor& t, const char* name) {
  if (t.dtype == GQA_BF16) return fail(GQA_ERR_UNSUPPORTED, "bfloat16 is not implemented");
  if (t.dtype != GQA_F32 && t.dtype != GQA_F16)
    return fail(GQA_ERR_INVALID_ARGUMENT, "%s dtype must be float32 or float16", name);
  return GQA_OK;
}

gqa_status check_head_size(long long H) {
  if (H % 16 != 0 || H < 16 || H > 256)
    return fail(GQA_ERR_UNSUPPORTED, "head_size %lld: supported head sizes are multiples of 16 in [16, 256]", H);
  return GQA_OK;
}

gqa_status check_status_word(const void* status) {
  if (reinterpret_cast<uintptr_t>(status) & 3u)
    return fail(GQA_ERR_INVALID_ARGUMENT, "status must be 4-byte aligned");
  return GQA_OK;
}

constexpr long long kElems = 1LL << 40;   // elements of a tensor (byte offsets stay far below 2^63)

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

gqa_status check_block_cache(const gqa_block_cache& c, const char* name, long long B, long long Nkv, long long H,
                             long long* C) {
  if (c.block_size != 16 && c.block_size != 32 && c.block_size != 64 && c.block_size != 128 && c.block_size != 256)
    return fail(GQA_ERR_INVALID_ARGUMENT, "%s: block_size must be 16, 32, 64, 128 or 256", name);
  if (!present(c.key_codes) || !present(c.value_codes) || !present(c.key_scales) || !present(c.value_scales))
    return fail(GQA_ERR_INVALID_ARGUMENT, "%s: codes and scales are required", name);
  const gqa_tensor& k = c.key_codes;
  if (k.dtype != GQA_I8 || k.ndim != 4 || k.shape[0] != B || k.shape[1] != Nkv || k.shape[2] < 1 || k.shape[3] != H ||
      c.value_codes.dtype != GQA_I8 || !shape_is(c.value_codes, 4, k.shape))
    return fail(GQA_ERR_INVALID_ARGUMENT,
                "%s: codes must be int8 (B, kv_num_heads, C, head_size) = (%lld,%lld,C,%lld)", name, B, Nkv, H);
  *C = k.shape[2];
  const int64_t ss[3] = {B, Nkv, (*C + c.block_size - 1) / c.block_size};
  for (const gqa_tensor* t : {&c.key_scales, &c.value_scales})
    if (t->dtype != GQA_F32 || !shape_is(*t, 3, ss))
      return fail(GQA_ERR_INVALID_ARGUMENT, "%s: scales must be float32 (B, kv_num_heads, ceil(C / block_size)) = (%lld,%lld,%lld)",
                  name, B, Nkv, (long long)ss[2]);
  if (*C > (1LL << 30) || B * Nkv > 65535 || B * Nkv * *C >= (1LL << 31))   // TMA rows are 32-bit
    return fail(GQA_ERR_UNSUPPORTED, "%s: tensor too large", name);
  return GQA_OK;
}

// Whether the tensor-core prefill takes a call, which its head size and group
// size allow, rather than the split over the keys. The prefill runs a CTA per
// 256 query rows of a KV head over their whole key range; few long ranges leave
// most SMs idle there, while the split gives every warp an equal share. Both are
// estimated from measurements (us; fp16, fp32, with a softcap): a wave of
// prefill CTAs takes 1.95, 3.6, 3.5 per 128 keys (0.95, fp32 1.1 times that for
// one query tile, whose softmax nothing runs beside), a worker of the split 2.1, 2.1, 3.6
// per 32 keys and row tile, its merge 0.003 per query row. Measured on both
// sides: 64 rows a head on 32768 keys 492 against 240 us, 256 rows on 2048 keys
// 43 against 96, 24 fp32 rows on 25000 keys 836 against 51.
bool use_prefill(const BlockParams& P) {
  const int live = P.S < P.T ? P.S : P.T;   // positions behind total_sequence_length are padding
  const long long rows = (long long)live * P.G;
  const int rt = gqa::block_row_tile(P.t_type, P.H, rows);
  const double nrt = (double)((rows + rt - 1) / rt), heads = (double)P.B * P.Nkv;
  const double ctas = heads * (double)((rows + 2 * P.tile_rows - 1) / (2 * P.tile_rows)), waves = ceil(ctas / 152.0);
  double mean = P.T - 0.5 * live, most = P.T;   // keys a query row sees
  if (P.window >= 0) {
    mean = mean < P.window ? mean : P.window;
    most = most < (double)P.window + P.S ? most : (double)P.window + P.S;
  }
  const bool f32 = P.t_type == gqa::kF32, cap = P.softcap > 0.f;
  double tile = f32 ? 3.6 : cap ? 3.5 : 1.95;
  if (rows <= P.tile_rows) tile *= f32 ? 1.1 : 0.95;
  const double prefill = 8.0 + waves * (waves > 1.0 ? mean : most) / 128.0 * tile;
  const double split = 10.0 + heads * nrt * (mean / 32.0 + 2.0) / 1216.0 * (cap ? 3.6 : 2.1) + heads * rows * 0.003;
  return prefill <= split;
}

struct BlockPlan {
  BlockParams P;
  bool prefill;                                // tensor-core prefill instead of the split over the keys
  size_t part_o, part_ml, stash, lse, o_acc, total;   // bytes of each section
};

gqa_status plan_block(const gqa_handle* h, const gqa_block_cache* cache, const gqa_block_inputs* in,
                      const gqa_block_outputs* out, BlockPlan* pl) {
  if (!h || !cache || !in || !out) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL handle, cache, inputs or outputs");
  const gqa_attrs& a = h->attrs;
  if (!a.causal) return fail(GQA_ERR_UNSUPPORTED, "attention over a block-scaled cache is causal");
  if (a.do_rotary) return fail(GQA_ERR_UNSUPPORTED, "do_rotary does not apply here: rotate with gqa_rotary_axes");
  if (a.k_quant_type != GQA_QUANT_NONE || a.v_quant_type != GQA_QUANT_NONE)
    return fail(GQA_ERR_UNSUPPORTED, "k/v_quant_type do not apply to a block-scaled cache");
  if (a.sliding_window_cache) return fail(GQA_ERR_UNSUPPORTED, "sliding_window_cache does not apply to a block-scaled cache");
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
  long long C = 0;
  if ((s = check_block_cache(*cache, "cache", B, Nkv, H, &C)) != GQA_OK) return s;
  if (present(in->key) != present(in->value)) return fail(GQA_ERR_INVALID_ARGUMENT, "key and value come together");
  const int64_t kvs[3] = {B, S, Nkv * H};
  for (const gqa_tensor* t : {&in->key, &in->value})
    if (present(*t) && (t->dtype != q.dtype || !shape_is(*t, 3, kvs)))
      return fail(GQA_ERR_INVALID_ARGUMENT, "key/value must be (B, S, kv_num_heads*head_size) of the query dtype");
  const int64_t b1[1] = {B};
  if (!present(in->seqlens_k) || in->seqlens_k.dtype != GQA_I32 || !shape_is(in->seqlens_k, 1, b1))
    return fail(GQA_ERR_INVALID_ARGUMENT, "seqlens_k must be int32 of shape (B)");
  if (present(in->new_lens) && (in->new_lens.dtype != GQA_I32 || !shape_is(in->new_lens, 1, b1)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "new_lens must be int32 of shape (B)");
  const int64_t n1[1] = {N};
  if (present(in->head_sink) && (in->head_sink.dtype != q.dtype || !shape_is(in->head_sink, 1, n1)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "head_sink must be (num_heads) of the query dtype");
  const int64_t ws[3] = {B, Nkv, C};
  for (const gqa_tensor* t : {&in->past_weights, &out->present_weights})
    if (present(*t) && (t->dtype != GQA_F32 || !shape_is(*t, 3, ws)))
      return fail(GQA_ERR_INVALID_ARGUMENT, "past/present_weights must be float32 (B, kv_num_heads, C)");
  if (present(in->past_weights) && !present(out->present_weights))
    return fail(GQA_ERR_INVALID_ARGUMENT, "past_weights needs present_weights");
  if (!present(out->output) || out->output.dtype != q.dtype || !shape_is(out->output, 3, q.shape))
    return fail(GQA_ERR_INVALID_ARGUMENT, "output must have the query's shape and dtype");
  const long long T = in->total_sequence_length;
  if (T < 1 || T > C) return fail(GQA_ERR_INVALID_ARGUMENT, "total_sequence_length %lld must be in [1, C = %lld]", T, C);
  if (S > C) return fail(GQA_ERR_INVALID_ARGUMENT, "sequence_length %lld exceeds the cache capacity %lld", S, C);
  const long long G = N / Nkv;
  if (S * N > (1LL << 30) || B * S * N > (1LL << 31) - 65536) return fail(GQA_ERR_UNSUPPORTED, "query too large");

  const Named read[] = {{&in->query, "query"}, {&in->key, "key"}, {&in->value, "value"}, {&in->seqlens_k, "seqlens_k"},
                        {&in->new_lens, "new_lens"}, {&in->head_sink, "head_sink"}, {&in->past_weights, "past_weights"}};
  const Named written[] = {{&cache->key_codes, "key_codes"}, {&cache->value_codes, "value_codes"},
                           {&cache->key_scales, "key_scales"}, {&cache->value_scales, "value_scales"},
                           {&out->output, "output"}, {&out->present_weights, "present_weights"}};
  const gqa_tensor* same[][2] = {{&out->present_weights, &in->past_weights}};
  if ((s = check_buffers(read, 7, written, 6, same, 1)) != GQA_OK) return s;

  BlockParams& P = pl->P;
  memset(&P, 0, sizeof(P));
  P.B = (int)B; P.S = (int)S; P.N = (int)N; P.Nkv = (int)Nkv; P.G = (int)G; P.H = (int)H;
  P.C = (int)C; P.T = (int)T;
  P.bs_log2 = log2_of(cache->block_size);
  P.nblk = (int)cache->key_scales.shape[2];
  P.t_type = q.dtype == GQA_F16 ? gqa::kF16 : gqa::kF32;
  // A window that reaches every row hides none; what remains is below 2^30, so the kernels' sums fit 32 bits.
  P.window = a.local_window_size < T ? a.local_window_size : -1;
  P.scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf((float)H);
  P.softcap = a.softcap;
  P.smooth = a.smooth_softmax == 1 ? 1 : 0;
  P.q = q.data; P.k = in->key.data; P.v = in->value.data;
  P.out = out->output.data;
  P.kc = static_cast<int8_t*>(cache->key_codes.data);
  P.vc = static_cast<int8_t*>(cache->value_codes.data);
  P.ks = static_cast<float*>(cache->key_scales.data);
  P.vs = static_cast<float*>(cache->value_scales.data);
  P.seqlens = static_cast<const int*>(in->seqlens_k.data);
  P.new_lens = static_cast<const int*>(in->new_lens.data);
  P.sink = in->head_sink.data;
  P.past_w = static_cast<const float*>(in->past_weights.data);
  P.present_w = static_cast<float*>(out->present_weights.data);
  P.wait_budget = h->wait_budget;
  P.withhold_tile = h->withhold_tile;

  const long long rows = S * G;
  // (The prefill takes row maxima and masks before the scale: a negative one would turn them.)
  P.tile_rows = G <= 128 ? (int)(128 / G * G) : 0;
  const long long nqb = G <= 128 ? (rows + 2 * P.tile_rows - 1) / (2 * P.tile_rows) : 0;
  const bool grid_ok = nqb <= 65535 && (T + 127) / 128 <= 65535;
  pl->prefill = H <= 128 && G <= 128 && P.scale > 0.f && rows > 16 && grid_ok && use_prefill(P);
  pl->part_o = pl->part_ml = pl->stash = pl->lse = pl->o_acc = 0;
  if (pl->prefill) {
    if (P.t_type == gqa::kF32 && T > gqa::kPrefillFlush)
      pl->o_acc = align_up((size_t)(B * Nkv) * nqb * 2 * 128 * 128 * sizeof(float));
    P.qb_major = 2 * S >= T;   // key ranges differ by query block more than by sequence
  } else {
    P.rt_rows = gqa::block_row_tile(P.t_type, (int)H, rows);
    P.nrt = (int)((rows + P.rt_rows - 1) / P.rt_rows);
    P.flush = P.t_type == gqa::kF32 && P.nrt > 1;
    P.workers = gqa::block_workers(P);
    const size_t slots = (size_t)P.workers + (size_t)(B * Nkv) * P.nrt;
    pl->part_o = align_up(slots * P.rt_rows * H * sizeof(float));
    pl->part_ml = align_up(slots * P.rt_rows * 4 * sizeof(float));   // m, l, l of the rounded probabilities, -
  }
  if (P.present_w) {
    if (!pl->prefill && P.nrt == 1) {
      P.stash_ld = (int)((T + gqa::kBlockUnit - 1) / gqa::kBlockUnit * gqa::kBlockUnit);
      P.stash_rows = (int)((rows + 1) & ~1LL);
      pl->stash = align_up((size_t)(B * Nkv) * P.stash_ld * P.stash_rows * sizeof(float));
    } else {
      pl->lse = align_up((size_t)(B * Nkv * rows) * sizeof(float));
    }
  }
  pl->total = pl->part_o + pl->part_ml + pl->stash + pl->lse + pl->o_acc;
  return GQA_OK;
}

}  // namespace

extern "C" {

gqa_status gqa_rotary_axes(gqa_handle* h, const gqa_rotary_inputs* in, const gqa_rotary_outputs* out, void* status,
                           void* stream) {
  if (!h || !in || !out) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL handle, inputs or outputs");
  gqa_status s;
  const gqa_tensor& q = in->query;
  if (!present(q)) return fail(GQA_ERR_INVALID_ARGUMENT, "query is required");
  if ((s = check_float(q, "query")) != GQA_OK) return s;
  if (q.ndim != 3 || q.shape[0] < 1 || q.shape[1] < 1 || q.shape[2] < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "query must be a non-empty (B, S, N*H)");
  const long long B = q.shape[0], S = q.shape[1], N = h->attrs.num_heads, Nkv = h->attrs.kv_num_heads;
  if (q.shape[2] % N) return fail(GQA_ERR_INVALID_ARGUMENT, "query hidden size %lld is not a multiple of num_heads %lld", (long long)q.shape[2], N);
  const long long H = q.shape[2] / N;
  if ((s = check_head_size(H)) != GQA_OK) return s;
  const int64_t ks[3] = {B, S, Nkv * H};
  if (present(in->key) && (in->key.dtype != q.dtype || !shape_is(in->key, 3, ks)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "key must be (B, S, kv_num_heads*head_size) of the query dtype");
  if (!present(out->query) || out->query.dtype != q.dtype || !shape_is(out->query, 3, q.shape))
    return fail(GQA_ERR_INVALID_ARGUMENT, "output query must have the query's shape and dtype");
  if (present(out->key) != present(in->key) ||
      (present(out->key) && (out->key.dtype != q.dtype || !shape_is(out->key, 3, ks))))
    return fail(GQA_ERR_INVALID_ARGUMENT, "output key must have the key's shape and dtype");
  const int A = in->num_axes;
  if (A < 1 || A > GQA_MAX_ROTARY_AXES)
    return fail(GQA_ERR_INVALID_ARGUMENT, "num_axes must be in [1, %d]", GQA_MAX_ROTARY_AXES);
  if (in->interleaved != 0 && in->interleaved != 1) return fail(GQA_ERR_INVALID_ARGUMENT, "interleaved must be 0 or 1");
  long long pairs = 0;
  for (int i = 0; i < A; ++i) {
    if (in->sections[i] < 0 || in->sections[i] > H) return fail(GQA_ERR_INVALID_ARGUMENT, "a section is outside [0, head_size / 2]");
    pairs += in->sections[i];
  }
  if (pairs < 1 || 2 * pairs > H)
    return fail(GQA_ERR_INVALID_ARGUMENT, "the sections add up to %lld pairs; head_size %lld has %lld", pairs, H, H / 2);
  if (pairs % 8) return fail(GQA_ERR_UNSUPPORTED, "the sum of the sections must be a multiple of 8");
  if (in->interleaved)
    for (int r = 1; r < A; ++r)
      if (in->sections[r] > 0 && (long long)(in->sections[r] - 1) * A + r >= pairs)
        return fail(GQA_ERR_INVALID_ARGUMENT, "interleaved section %d does not fit among %lld pairs", r, pairs);
  const int64_t ps[3] = {A, B, S};
  if (!present(in->positions) || in->positions.dtype != GQA_I32 || !shape_is(in->positions, 3, ps))
    return fail(GQA_ERR_INVALID_ARGUMENT, "positions must be int32 (num_axes, B, S)");
  const gqa_tensor& c = in->cos_cache;
  if (!present(c) || !present(in->sin_cache) || (c.dtype != q.dtype && c.dtype != GQA_F32) || c.ndim != 2 ||
      c.shape[0] < 1 || c.shape[0] >= (1LL << 31) || c.shape[1] != pairs || in->sin_cache.dtype != c.dtype ||
      !shape_is(in->sin_cache, 2, c.shape))
    return fail(GQA_ERR_INVALID_ARGUMENT, "cos/sin_cache must be (R, %lld), both of the query dtype or both float32", pairs);
  const int64_t h1[1] = {H};
  const bool qn = present(in->q_norm_weight), kn = present(in->k_norm_weight);
  if (present(in->key) ? qn != kn : kn)
    return fail(GQA_ERR_INVALID_ARGUMENT, "q_norm_weight and k_norm_weight must be given together (q_norm_weight alone without a key)");
  for (const gqa_tensor* t : {&in->q_norm_weight, &in->k_norm_weight})
    if (present(*t) && (t->dtype != q.dtype || !shape_is(*t, 1, h1)))
      return fail(GQA_ERR_INVALID_ARGUMENT, "q/k_norm_weight must be (head_size) of the query dtype");
  if (N * H > (1LL << 30))   // a token's coordinates are counted in 32 bits
    return fail(GQA_ERR_UNSUPPORTED, "query hidden size %lld: at most 2^30", N * H);
  if (B * S > (1LL << 31) || B * S > kElems / (N * H)) return fail(GQA_ERR_UNSUPPORTED, "query too large");
  if ((s = check_status_word(status)) != GQA_OK) return s;
  const Named read[] = {{&in->query, "query"}, {&in->key, "key"}, {&in->positions, "positions"}, {&in->cos_cache, "cos_cache"},
                        {&in->sin_cache, "sin_cache"}, {&in->q_norm_weight, "q_norm_weight"}, {&in->k_norm_weight, "k_norm_weight"}};
  const Named written[] = {{&out->query, "output query"}, {&out->key, "output key"}};
  const gqa_tensor* same[][2] = {{&out->query, &in->query}, {&out->key, &in->key}};
  if ((s = check_buffers(read, 7, written, 2, same, 2)) != GQA_OK) return s;

  gqa::RotaryAxesParams P;
  memset(&P, 0, sizeof(P));
  P.q = q.data; P.k = in->key.data; P.qo = out->query.data; P.ko = out->key.data;
  P.pos = static_cast<const int*>(in->positions.data);
  P.cos_c = c.data; P.sin_c = in->sin_cache.data;
  P.qw = in->q_norm_weight.data; P.kw = in->k_norm_weight.data;
  P.status = static_cast<uint32_t*>(status);
  P.tokens = B * S;
  P.N = (int)N; P.Nkv = (int)Nkv; P.H = (int)H; P.pairs = (int)pairs; P.table_rows = (int)c.shape[0];
  P.table_f32 = c.dtype == GQA_F32 ? 1 : 0;
  P.eps = h->attrs.qk_norm_epsilon;
  for (int l = 0; l < (int)pairs / 8; ++l) {
    unsigned nib = 0;
    bool uniform = true;
    for (int e = 0; e < 8; ++e) {
      const int d = 8 * l + e;
      int axis = 0;
      if (in->interleaved) {
        const int r = d % A;
        axis = r > 0 && d < A * in->sections[r] ? r : 0;
      } else {
        for (int end = in->sections[0]; d >= end; end += in->sections[axis]) ++axis;
      }
      nib |= (unsigned)axis << (4 * e);
      uniform = uniform && (unsigned)axis == (nib & 15u);
    }
    P.axis_nibbles[l] = nib;
    P.chunk_uniform[l] = uniform;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed_launch(h, GQA_KERNEL_ROTARY_AXES, st, [&] {
    return gqa::launch_rotary_axes(P, q.dtype == GQA_F16 ? gqa::kF16 : gqa::kF32, st);
  });
  return e == cudaSuccess ? GQA_OK : cuda_fail(e, "rotary launch");
}

gqa_status gqa_block_workspace_size(const gqa_handle* h, const gqa_block_cache* cache, const gqa_block_inputs* in,
                                    const gqa_block_outputs* out, size_t* bytes) {
  if (!bytes) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL bytes pointer");
  BlockPlan pl;
  gqa_status s = plan_block(h, cache, in, out, &pl);
  if (s != GQA_OK) return s;
  *bytes = pl.total;
  return GQA_OK;
}

gqa_status gqa_block_describe_plan(const gqa_handle* h, const gqa_block_cache* cache, const gqa_block_inputs* in,
                                   const gqa_block_outputs* out, gqa_plan_info* info) {
  if (!info) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL info pointer");
  BlockPlan pl;
  gqa_status s = plan_block(h, cache, in, out, &pl);
  if (s != GQA_OK) return s;
  info->regime = pl.prefill ? GQA_REGIME_PREFILL : GQA_REGIME_DECODE;
  info->launches = (pl.P.k ? 1 : 0) + (pl.prefill ? 1 : 2) + (pl.lse ? 1 : 0);
  info->split_len = pl.prefill ? 0 : gqa::kBlockUnit;
  info->max_splits = pl.prefill ? 0 : pl.P.workers;
  info->workspace_bytes = pl.total;
  return GQA_OK;
}

gqa_status gqa_block_forward(gqa_handle* h, const gqa_block_cache* cache, const gqa_block_inputs* in,
                             const gqa_block_outputs* out, void* ws, size_t ws_bytes, void* status, void* stream) {
  BlockPlan pl;
  gqa_status s = plan_block(h, cache, in, out, &pl);
  if (s != GQA_OK) return s;
  if ((s = check_status_word(status)) != GQA_OK) return s;
  if (pl.total && (!ws || (reinterpret_cast<uintptr_t>(ws) % gqa::kAlign) != 0))
    return fail(GQA_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (ws_bytes < pl.total) return fail(GQA_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, pl.total);
  BlockParams& P = pl.P;
  char* w = static_cast<char*>(ws);
  P.part_o = reinterpret_cast<float*>(w);
  P.part_ml = reinterpret_cast<float*>(w + pl.part_o);
  if (pl.stash) P.stash = reinterpret_cast<float*>(w + pl.part_o + pl.part_ml);
  if (pl.lse) P.lse = reinterpret_cast<float*>(w + pl.part_o + pl.part_ml);
  if (pl.o_acc) P.o_acc = reinterpret_cast<float*>(w + pl.part_o + pl.part_ml + pl.lse);
  P.status = static_cast<uint32_t*>(status);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (P.k) {
    e = timed_launch(h, GQA_KERNEL_BLOCK_APPEND, st, [&] { return gqa::launch_block_append(P, st); });
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
  }
  if (pl.prefill) {
    e = timed_launch(h, GQA_KERNEL_BLOCK_PREFILL, st, [&] { return gqa::launch_block_prefill(P, st); });
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
  } else {
    e = timed_launch(h, GQA_KERNEL_BLOCK_ATTENTION, st, [&] { return gqa::launch_block_attn(P, st); });
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
    e = timed_launch(h, GQA_KERNEL_BLOCK_MERGE, st, [&] { return gqa::launch_block_merge(P, st); });
    if (e != cudaSuccess) return cuda_fail(e, "merge launch");
  }
  if (P.lse) {
    e = timed_launch(h, GQA_KERNEL_BLOCK_WEIGHTS, st, [&] {
      const bool tc = pl.prefill && P.t_type == gqa::kF16 && (P.G <= 64 || P.G == 128);
      return tc ? gqa::launch_block_weights_tc(P, st) : gqa::launch_block_weights(P, st);
    });
    if (e != cudaSuccess) return cuda_fail(e, "weights launch");
  }
  return GQA_OK;
}

gqa_status gqa_block_evict(gqa_handle* h, const gqa_evict_args* a, void* status, void* stream) {
  if (!h || !a) return fail(GQA_ERR_INVALID_ARGUMENT, "NULL handle or arguments");
  const gqa_tensor& k = a->from.key_codes;
  if (!present(k) || k.ndim != 4 || k.shape[0] < 1 || k.shape[3] < 1)
    return fail(GQA_ERR_INVALID_ARGUMENT, "from: codes must be int8 (B, kv_num_heads, C, head_size)");
  const long long B = k.shape[0], Nkv = h->attrs.kv_num_heads, H = k.shape[3];
  gqa_status s;
  if ((s = check_head_size(H)) != GQA_OK) return s;
  long long C = 0, Cto = 0;
  if ((s = check_block_cache(a->from, "from", B, Nkv, H, &C)) != GQA_OK) return s;
  if ((s = check_block_cache(a->into, "into", B, Nkv, H, &Cto)) != GQA_OK) return s;
  if (a->from.block_size != a->into.block_size)
    return fail(GQA_ERR_INVALID_ARGUMENT, "from and into must have one block_size");
  const long long T = a->total_sequence_length, keep = a->keep;
  if (T < 1 || T > C) return fail(GQA_ERR_INVALID_ARGUMENT, "total_sequence_length %lld must be in [1, C = %lld]", T, C);
  if (keep < 1 || a->recent < 0 || a->first < 0 || (long long)a->recent + a->first > keep)
    return fail(GQA_ERR_INVALID_ARGUMENT, "keep must be positive, first and recent not negative, and first + recent at most keep");
  if (Cto < (keep < T ? keep : T))
    return fail(GQA_ERR_INVALID_ARGUMENT, "into holds %lld rows; min(keep, total_sequence_length) = %lld are needed", Cto, keep < T ? keep : T);
  if (keep > (1LL << 30)) return fail(GQA_ERR_UNSUPPORTED, "keep too large");
  if (a->fill_skipped & ~(GQA_FILL_KEPT | GQA_FILL_SEQLENS)) return fail(GQA_ERR_INVALID_ARGUMENT, "unknown fill_skipped bits");
  const int64_t ws[3] = {B, Nkv, C}, wt[3] = {B, Nkv, Cto}, kp[3] = {B, Nkv, keep}, b1[1] = {B};
  if (!present(a->weights) || a->weights.dtype != GQA_F32 || !shape_is(a->weights, 3, ws))
    return fail(GQA_ERR_INVALID_ARGUMENT, "weights must be float32 (B, kv_num_heads, C)");
  if (present(a->into_weights) && (a->into_weights.dtype != GQA_F32 || !shape_is(a->into_weights, 3, wt)))
    return fail(GQA_ERR_INVALID_ARGUMENT, "into_weights must be float32 (B, kv_num_heads, C of into)");
  if (!present(a->kept) || a->kept.dtype != GQA_I32 || !shape_is(a->kept, 3, kp))
    return fail(GQA_ERR_INVALID_ARGUMENT, "kept must be int32 (B, kv_num_heads, keep)");
  for (const gqa_tensor* t : {&a->seqlens_k, &a->into_seqlens_k})
    if (!present(*t) || t->dtype != GQA_I32 || !shape_is(*t, 1, b1))
      return fail(GQA_ERR_INVALID_ARGUMENT, "seqlens_k and into_seqlens_k must be int32 of shape (B)");
  if ((s = check_status_word(status)) != GQA_OK) return s;
  const Named read[] = {{&a->from.key_codes, "from key_codes"}, {&a->from.value_codes, "from value_codes"},
                        {&a->from.key_scales, "from key_scales"}, {&a->from.value_scales, "from value_scales"},
                        {&a->weights, "weights"}, {&a->seqlens_k, "seqlens_k"}};
  const Named written[] = {{&a->into.key_codes, "into key_codes"}, {&a->into.value_codes, "into value_codes"},
                           {&a->into.key_scales, "into key_scales"}, {&a->into.value_scales, "into value_scales"},
                           {&a->into_weights, "into_weights"}, {&a->kept, "kept"}, {&a->into_seqlens_k, "into_seqlens_k"}};
  if ((s = check_buffers(read, 6, written, 7, nullptr, 0)) != GQA_OK) return s;

  gqa::EvictParams P;
  memset(&P, 0, sizeof(P));
  P.B = (int)B; P.Nkv = (int)Nkv; P.H = (int)H; P.C = (int)C; P.Cto = (int)Cto; P.T = (int)T;
  P.bs_log2 = log2_of(a->from.block_size);
  P.nblk = (int)a->from.key_scales.shape[2];
  P.nblk_to = (int)a->into.key_scales.shape[2];
  P.keep = a->keep; P.recent = a->recent; P.first = a->first;
  P.fill = a->fill_skipped;
  P.kc = static_cast<const int8_t*>(a->from.key_codes.data);
  P.vc = static_cast<const int8_t*>(a->from.value_codes.data);
  P.ks = static_cast<const float*>(a->from.key_scales.data);
  P.vs = static_cast<const float*>(a->from.value_scales.data);
  P.kc_to = static_cast<int8_t*>(a->into.key_codes.data);
  P.vc_to = static_cast<int8_t*>(a->into.value_codes.data);
  P.ks_to = static_cast<float*>(a->into.key_scales.data);
  P.vs_to = static_cast<float*>(a->into.value_scales.data);
  P.w = static_cast<const float*>(a->weights.data);
  P.w_to = static_cast<float*>(a->into_weights.data);
  P.seqlens = static_cast<const int*>(a->seqlens_k.data);
  P.kept = static_cast<int*>(a->kept.data);
  P.seqlens_to = static_cast<int*>(a->into_seqlens_k.data);
  P.status = static_cast<uint32_t*>(status);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed_launch(h, GQA_KERNEL_EVICT_SELECT, st, [&] { return gqa::launch_evict_select(P, st); });
  if (e != cudaSuccess) return cuda_fail(e, "selection launch");
  e = timed_launch(h, GQA_KERNEL_EVICT_GATHER, st, [&] { return gqa::launch_evict_gather(P, st); });
  return e == cudaSuccess ? GQA_OK : cuda_fail(e, "gather launch");
}

}  // extern "C"
