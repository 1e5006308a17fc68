// Host side of the operators on token caches: argument checks, translation of
// the public descriptors into launch parameters, and the exported C entry
// points.
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "kda_cache.hpp"
#include "kda_host.hpp"
#include "kda_recoverssm.h"

using namespace kda::host;

namespace {

constexpr int64_t kI32Max = 0x7fffffff;
constexpr int64_t kMaxThreads = 0xffffffff;   // work items of a launch
constexpr int64_t kMaxGroups = kMaxThreads / 256;
constexpr float kLog2e = 1.44269504088896340736f;

// Strides of a tensor of 16-byte aligned rows (its last dimension).
int check_rows(const kda_tensor& t, const char* name) {
  const int last = t.ndim - 1, es = elem_size(t.dtype);
  if (t.shape[last] > 1 && t.stride[last] != 1)
    return fail(KDA_E_LAYOUT, "%s must have contiguous rows", name);
  bool rows = true;
  for (int i = 0; i < last; ++i) {
    if (t.shape[i] <= 1) continue;
    if (t.stride[i] < 0)
      return fail(KDA_E_LAYOUT, "%s has a negative stride", name);
    rows &= t.stride[i] * es % 16 == 0;
  }
  if (!rows || !aligned(t.data, 16))
    return fail(KDA_E_UNALIGNED, "a row of %s does not start on a 16-byte "
                "boundary", name);
  return KDA_OK;
}

// Whether every element has a place of its own: each dimension's stride past
// the extent of those of smaller stride.
bool apart(const kda_tensor& t) {
  int order[4] = {0, 1, 2, 3};
  std::sort(order, order + t.ndim,
            [&](int i, int j) { return t.stride[i] < t.stride[j]; });
  int64_t extent = 0;          // from the first element to the last
  for (int k = 0; k < t.ndim; ++k) {
    const int i = order[k];
    if (t.shape[i] == 0) return true;
    if (t.shape[i] == 1) continue;
    if (t.stride[i] <= extent) return false;
    extent += (t.shape[i] - 1) * t.stride[i];
  }
  return true;
}

int check_cache(const kda_tensor& t) {
  KDA_TRY(check_desc(t, "cache", 3));
  if (t.shape[0] < 1 || t.shape[1] < 1)
    return fail(KDA_E_SHAPE, "the cache must be [blocks, block_size, dims]");
  if (t.shape[0] > kI32Max || t.shape[1] > kI32Max)
    return fail(KDA_E_CAPACITY, "the cache's blocks exceed 2^31");
  return check_rows(t, "cache");
}

// The kernels take scales above 0: queries are negated for one below, and a
// scale of 0 is one that leaves no difference between scores.
template <class Params>
int set_scale(float scale, Params* p) {
  p->negate = scale < 0.0f;
  p->scale = (scale < 0.0f ? -scale : scale) * kLog2e;
  if (!std::isfinite(p->scale))
    return fail(KDA_E_ARG, "softmax_scale must be finite");
  if (p->scale == 0.0f) p->scale = 0x1p-126f;
  return KDA_OK;
}

bool latent_dims(int64_t R, int64_t P) {
  return (R == 128 || R == 256 || R == 512) && (P == 0 || P == 64);
}

int plan_latent_write(const kda_latent_write_args* a,
                      kda::LatentWriteParams* p) {
  if (a == nullptr) return fail(KDA_E_ARG, "cache write arguments are NULL");
  KDA_TRY(check_cache(a->cache));
  KDA_TRY(check_desc(a->latent, "latent", 2));
  const kda_tensor &lat = a->latent, &rope = a->rope_key, &cache = a->cache;
  const int64_t T = lat.shape[0], W = cache.shape[2];
  const bool has_rope = rope.ndim != 0;
  const int es = elem_size(cache.dtype);
  if (has_rope) KDA_TRY(check_desc(rope, "rope_key", 2));
  if (lat.dtype != cache.dtype || (has_rope && rope.dtype != cache.dtype))
    return fail(KDA_E_DTYPE,
                "latent, rope_key and cache must share one dtype");
  const int64_t P = has_rope ? rope.shape[1] : 0;
  if ((has_rope && rope.shape[0] != T) || lat.shape[1] + P != W ||
      lat.shape[1] < 1)
    return fail(KDA_E_SHAPE,
                "latent [T, R] and rope_key [T, P] must fill the cache's "
                "R + P = %lld values",
                (long long)W);
  if (lat.shape[1] * es % 16 != 0 || P * es % 16 != 0)
    return fail(KDA_E_UNSUPPORTED,
                "latent and rope key take multiples of 16 bytes");
  KDA_TRY(check_rows(lat, "latent"));
  if (has_rope) KDA_TRY(check_rows(rope, "rope_key"));
  if (!apart(cache)) return fail(KDA_E_LAYOUT, "the cache's entries overlap");
  if (a->null_block_id < 0)
    return fail(KDA_E_ARG, "null_block_id must not be negative");
  if (T > kI32Max || T * (W * es / 16) > kMaxThreads - 256)
    return fail(KDA_E_CAPACITY, "too many tokens");
  if (T > 0 && !a->slot_mapping)
    return fail(KDA_E_ARG, "slot_mapping is required");
  if (!aligned(a->slot_mapping, 8))
    return fail(KDA_E_UNALIGNED, "slot_mapping must be 8-byte aligned");
  *p = kda::LatentWriteParams{};
  p->latent = static_cast<const char*>(lat.data);
  p->rope = static_cast<const char*>(rope.data);
  p->s_lat = lat.stride[0] * es;
  p->s_rope = has_rope ? rope.stride[0] * es : 0;
  p->cache = static_cast<char*>(cache.data);
  p->s_blk = cache.stride[0] * es;
  p->s_tok = cache.stride[1] * es;
  p->slots = a->slot_mapping;
  p->total_slots = cache.shape[0] * cache.shape[1];
  p->first_slot = (int64_t(a->null_block_id) + 1) * cache.shape[1];
  p->T = int32_t(T);
  p->block = int32_t(cache.shape[1]);
  p->lat_chunks = int32_t(lat.shape[1] * es / 16);
  p->chunks = int32_t(W * es / 16);
  return KDA_OK;
}

// A cache seen through request rows and a block table.
template <class Args>
int plan_paged(const Args* a, const kda_tensor& cache, kda::PagedParams* p) {
  if (a->batch < 0 || a->num_request_rows < 0 || a->block_table_width < 0)
    return fail(KDA_E_ARG, "a count is negative");
  if (a->null_block_id < 0)
    return fail(KDA_E_ARG, "null_block_id must not be negative");
  const int64_t sr = a->block_table_strides[0], sc = a->block_table_strides[1];
  if (sr < 0 || sc < 0 || sr > kI32Max || sc > kI32Max)
    return fail(KDA_E_LAYOUT, "a table stride is negative or exceeds 2^31");
  if (a->num_request_rows > 0 && a->block_table_width > 0 && !a->block_table)
    return fail(KDA_E_ARG, "block_table is required");
  if (!aligned(a->block_table, 4) || !aligned(a->request_indices, 4))
    return fail(KDA_E_UNALIGNED, "metadata pointers must be 4-byte aligned");
  const int es = elem_size(cache.dtype);
  *p = kda::PagedParams{};
  p->req_idx = a->request_indices;
  p->table = a->block_table;
  p->s_tab_row = sr;
  p->s_tab_col = sc;
  p->cache = static_cast<const char*>(cache.data);
  p->s_blk = cache.stride[0] * es;
  p->s_tok = cache.stride[1] * es;
  p->B = a->batch;
  p->rows = a->num_request_rows;
  p->width = a->block_table_width;
  p->block = int32_t(cache.shape[1]);
  p->null_id = a->null_block_id;
  p->N = cache.shape[0];
  // magic = ceil(2^(31 + l) / block), 2^l the power of two not below block: at
  // most 2^32 - 1, and its error, below 1, times a position stays below 2^31
  int l = 0;
  while ((int64_t(1) << l) < p->block) ++l;
  p->shift = 31 + l;
  p->magic = uint32_t(((uint64_t(1) << p->shift) + p->block - 1) / p->block);
  return KDA_OK;
}

int64_t latent_bytes(int64_t T, int64_t B, int64_t H, int64_t R, int64_t P) {
  if (T < 0 || B < 0 || H < 1 || B > kI32Max || T > kI32Max ||
      H > kI32Max || T * H > kI32Max - 256 || !latent_dims(R, P))
    return 0;
  return kda::latent_work_bytes(kda::latent_groups(T, B, H), int(R));
}

struct LatentPlan {
  kda::LatentParams p;
  int R = 0, P = 0;
  bool bf16 = false, noop = false;
};

// lse: F32 [T, H] in any strides, or empty.
int check_lse(const kda_tensor& lse, int64_t T, int64_t H) {
  if (lse.ndim == 0) return KDA_OK;
  KDA_TRY(check_desc(lse, "lse", 2));
  if (lse.dtype != KDA_F32)
    return fail(KDA_E_DTYPE, "lse must be float32");
  if (!shape_is(lse, T, H))
    return fail(KDA_E_SHAPE, "lse must be [T, H]");
  if (lse.stride[0] < 0 || lse.stride[1] < 0 || !apart(lse))
    return fail(KDA_E_LAYOUT, "lse's entries overlap");
  if (!aligned(lse.data, 4))
    return fail(KDA_E_UNALIGNED, "lse must be 4-byte aligned");
  return KDA_OK;
}

int plan_latent(const kda_latent_args* a, LatentPlan* plan) {
  if (a == nullptr) return fail(KDA_E_ARG, "attention arguments are NULL");
  kda::LatentParams& p = plan->p;
  KDA_TRY(check_cache(a->cache));
  KDA_TRY(check_desc(a->q, "q", 3));
  KDA_TRY(check_desc(a->out, "out", 3));
  const int32_t act = a->q.dtype;
  if (a->cache.dtype != act || a->out.dtype != act)
    return fail(KDA_E_DTYPE, "q, cache and out must share one dtype");
  const int64_t T = a->q.shape[0], H = a->q.shape[1], W = a->q.shape[2];
  const int64_t R = a->out.shape[2], P = W - R;
  if (H < 1) return fail(KDA_E_SHAPE, "q must be [T, heads, R + P]");
  if (a->out.shape[0] != T || a->out.shape[1] != H || a->cache.shape[2] != W)
    return fail(KDA_E_SHAPE,
                "q [T, H, R + P], out [T, H, R] and cache [N, block, R + P] "
                "do not fit each other");
  if (!latent_dims(R, P))
    return fail(KDA_E_UNSUPPORTED,
                "latent dims 128, 256 and 512 and rope dims 0 and 64 are "
                "supported (got %lld and %lld)",
                (long long)R, (long long)P);
  KDA_TRY(check_rows(a->q, "q"));
  KDA_TRY(check_rows(a->out, "out"));
  if (!apart(a->out)) return fail(KDA_E_LAYOUT, "out's rows overlap");
  KDA_TRY(check_lse(a->lse, T, H));
  KDA_TRY(plan_paged(a, a->cache, &p.c));
  const bool bf16 = act == KDA_BF16;
  const int64_t need = latent_bytes(T, a->batch, H, R, P);
  if (need == 0)
    return fail(KDA_E_CAPACITY, "tokens and heads exceed 2^31 rows");
  plan->noop = a->batch == 0 || T == 0;
  if (!plan->noop) {
    if (!a->query_start_loc ||
        (a->num_request_rows > 0 && !a->num_computed_tokens))
      return fail(KDA_E_ARG,
                  "query_start_loc and num_computed_tokens are required");
    if (!aligned(a->query_start_loc, 4) ||
        !aligned(a->num_computed_tokens, 4))
      return fail(KDA_E_UNALIGNED,
                  "metadata pointers must be 4-byte aligned");
    if (!a->workspace) return fail(KDA_E_ARG, "the workspace is required");
    if (a->workspace_bytes < need)
      return fail(KDA_E_CAPACITY,
                  "the workspace holds %lld bytes; this attention needs %lld",
                  (long long)a->workspace_bytes, (long long)need);
    if (!aligned(a->workspace, 16))
      return fail(KDA_E_UNALIGNED, "the workspace must be 16-byte aligned");
  }
  const int es = elem_size(act);
  p.c.qsl = a->query_start_loc;
  p.c.computed = a->num_computed_tokens;
  p.q = static_cast<const char*>(a->q.data);
  p.s_q_tok = a->q.stride[0] * es;
  p.s_q_head = a->q.stride[1] * es;
  p.out = static_cast<char*>(a->out.data);
  p.s_out_tok = a->out.stride[0] * es;
  p.s_out_head = a->out.stride[1] * es;
  p.lse = a->lse.ndim ? static_cast<float*>(a->lse.data) : nullptr;
  p.s_lse_tok = a->lse.stride[0];
  p.s_lse_head = a->lse.stride[1];
  p.work = static_cast<char*>(a->workspace);
  KDA_TRY(set_scale(a->softmax_scale, &p));
  p.T = int32_t(T);
  p.H = int32_t(H);
  p.group = kda::latent_groups(T, a->batch, H);
  p.workers = kda::latent_workers(
      T, a->batch, H, int64_t(a->block_table_width) * a->cache.shape[1],
      p.group);
  plan->R = int(R);
  plan->P = int(P);
  plan->bf16 = bf16;
  return KDA_OK;
}

// key and value [S, H, D] of one dtype, rope_key [S, P] or empty.
int check_keys(const kda_tensor& key, const kda_tensor& value,
               const kda_tensor& rope, int64_t P) {
  KDA_TRY(check_desc(key, "key", 3));
  KDA_TRY(check_desc(value, "value", 3));
  const int64_t S = key.shape[0], H = key.shape[1], D = key.shape[2];
  if (value.dtype != key.dtype)
    return fail(KDA_E_DTYPE, "key and value must share one dtype");
  if (H < 1 || !shape_is(value, S, H, D))
    return fail(KDA_E_SHAPE, "key and value must be [S, heads, D]");
  if (D != 64 && D != 128)
    return fail(KDA_E_UNSUPPORTED, "head dims 64 and 128 are supported "
                "(got %lld)", (long long)D);
  KDA_TRY(check_rows(key, "key"));
  KDA_TRY(check_rows(value, "value"));
  if (rope.ndim == 0) return KDA_OK;
  KDA_TRY(check_desc(rope, "rope_key", 2));
  if (rope.dtype != key.dtype)
    return fail(KDA_E_DTYPE, "key and rope_key must share one dtype");
  if (!shape_is(rope, S, P))
    return fail(KDA_E_SHAPE, "rope_key must be [S, P] = [%lld, %lld]",
                (long long)S, (long long)P);
  return P > 0 ? check_rows(rope, "rope_key") : KDA_OK;
}

int plan_expand(const kda_latent_expand_args* a, kda::ExpandParams* p,
                bool* bf16) {
  if (a == nullptr) return fail(KDA_E_ARG, "expansion arguments are NULL");
  KDA_TRY(check_cache(a->cache));
  KDA_TRY(check_desc(a->weight, "weight", 3));
  const kda_tensor& w = a->weight;
  const int64_t R = w.shape[2], P = a->cache.shape[2] - R;
  KDA_TRY(check_keys(a->key, a->value, a->rope_key, P));
  const int64_t S = a->key.shape[0], H = a->key.shape[1], D = a->key.shape[2];
  if (a->cache.dtype != a->key.dtype || w.dtype != a->key.dtype)
    return fail(KDA_E_DTYPE,
                "cache, weight, key and value must share one dtype");
  if (!shape_is(w, H, 2 * D, R) || P < 0)
    return fail(KDA_E_SHAPE,
                "weight must be [H, 2 D, R] = [%lld, %lld, R <= %lld]",
                (long long)H, (long long)(2 * D),
                (long long)a->cache.shape[2]);
  const int es = elem_size(w.dtype);
  if (!latent_dims(R, 0) || P * es % 16 != 0)
    return fail(KDA_E_UNSUPPORTED,
                "latent dims 128, 256 and 512 and rope dims of a multiple of "
                "16 bytes are supported (got %lld and %lld)",
                (long long)R, (long long)P);
  KDA_TRY(check_rows(w, "weight"));
  if (!apart(a->key) || !apart(a->value) ||
      (a->rope_key.ndim && !apart(a->rope_key)))
    return fail(KDA_E_LAYOUT, "rows of key, value or rope_key overlap");
  KDA_TRY(plan_paged(a, a->cache, &p->c));
  if (S > kI32Max - 256 || H > kI32Max / 256 ||
      (H * 2 * D + 127) / 128 > 65535 ||
      (S + 127) / 128 * ((H * 2 * D + 127) / 128) > kMaxThreads / 256)
    return fail(KDA_E_CAPACITY, "key rows and heads exceed the grid");
  if (a->batch > 0 && S > 0 && !a->key_start_loc)
    return fail(KDA_E_ARG, "key_start_loc is required");
  if (!aligned(a->key_start_loc, 4))
    return fail(KDA_E_UNALIGNED, "metadata pointers must be 4-byte aligned");
  p->c.qsl = a->key_start_loc;
  p->w = static_cast<const char*>(w.data);
  p->s_w_head = w.stride[0] * es;
  p->s_w_row = w.stride[1] * es;
  p->key = static_cast<char*>(a->key.data);
  p->s_k_tok = a->key.stride[0] * es;
  p->s_k_head = a->key.stride[1] * es;
  p->value = static_cast<char*>(a->value.data);
  p->s_v_tok = a->value.stride[0] * es;
  p->s_v_head = a->value.stride[1] * es;
  p->rope = static_cast<char*>(a->rope_key.data);
  p->s_rope = a->rope_key.stride[0] * es;
  p->S = int32_t(S);
  p->H = int32_t(H);
  p->D = int32_t(D);
  p->R = int32_t(R);
  p->rope_chunks = a->rope_key.ndim ? int32_t(P * es / 16) : 0;
  *bf16 = w.dtype == KDA_BF16;
  return KDA_OK;
}

struct PromptPlan {
  kda::PromptParams p;
  int D = 0, P = 0;
  bool bf16 = false, noop = false;
};

int plan_prompt(const kda_latent_prefill_args* a, PromptPlan* plan) {
  if (a == nullptr)
    return fail(KDA_E_ARG, "prompt attention arguments are NULL");
  KDA_TRY(check_desc(a->q, "q", 3));
  KDA_TRY(check_desc(a->out, "out", 3));
  const int64_t T = a->q.shape[0], H = a->q.shape[1];
  const int64_t D = a->out.shape[2], P = a->q.shape[2] - D;
  const int32_t act = a->q.dtype;
  KDA_TRY(check_keys(a->key, a->value, a->rope_key, P));
  if (a->key.dtype != act || a->out.dtype != act)
    return fail(KDA_E_DTYPE, "q, key, value and out must share one dtype");
  if (H < 1 || !shape_is(a->out, T, H) || a->key.shape[1] != H ||
      a->key.shape[2] != D)
    return fail(KDA_E_SHAPE,
                "q [T, H, D + P], out [T, H, D] and key [S, H, D] do not fit "
                "each other");
  if (P != 0 && P != 64)
    return fail(KDA_E_UNSUPPORTED, "rope dims 0 and 64 are supported (got "
                "%lld)", (long long)P);
  if ((P > 0) != (a->rope_key.ndim != 0))
    return fail(KDA_E_SHAPE, "rope_key goes with q's last %lld values",
                (long long)P);
  KDA_TRY(check_rows(a->q, "q"));
  KDA_TRY(check_rows(a->out, "out"));
  if (!apart(a->out)) return fail(KDA_E_LAYOUT, "out's rows overlap");
  KDA_TRY(check_lse(a->lse, T, H));
  if (a->batch < 0) return fail(KDA_E_ARG, "batch is negative");
  const int64_t S = a->key.shape[0];
  if (T > kI32Max - 512 || S > kI32Max - 512 || H > kI32Max ||
      kda::prompt_tiles(T, a->batch) > kMaxThreads / 512 / H)
    return fail(KDA_E_CAPACITY, "tokens, requests and heads exceed the grid");
  plan->noop = T == 0 || a->batch == 0;
  if (!plan->noop && (!a->query_start_loc || !a->key_start_loc))
    return fail(KDA_E_ARG,
                "query_start_loc and key_start_loc are required");
  if (!aligned(a->query_start_loc, 4) || !aligned(a->key_start_loc, 4))
    return fail(KDA_E_UNALIGNED, "metadata pointers must be 4-byte aligned");
  const int es = elem_size(act);
  kda::PromptParams& p = plan->p;
  p = kda::PromptParams{};
  p.q = static_cast<const char*>(a->q.data);
  p.s_q_tok = a->q.stride[0] * es;
  p.s_q_head = a->q.stride[1] * es;
  p.key = static_cast<const char*>(a->key.data);
  p.s_k_tok = a->key.stride[0] * es;
  p.s_k_head = a->key.stride[1] * es;
  p.value = static_cast<const char*>(a->value.data);
  p.s_v_tok = a->value.stride[0] * es;
  p.s_v_head = a->value.stride[1] * es;
  p.rope = static_cast<const char*>(a->rope_key.data);
  p.s_rope = a->rope_key.stride[0] * es;
  p.out = static_cast<char*>(a->out.data);
  p.s_out_tok = a->out.stride[0] * es;
  p.s_out_head = a->out.stride[1] * es;
  p.lse = a->lse.ndim ? static_cast<float*>(a->lse.data) : nullptr;
  p.s_lse_tok = a->lse.stride[0];
  p.s_lse_head = a->lse.stride[1];
  p.qsl = a->query_start_loc;
  p.ksl = a->key_start_loc;
  KDA_TRY(set_scale(a->softmax_scale, &p));
  p.T = int32_t(T);
  p.S = int32_t(S);
  p.H = int32_t(H);
  p.B = a->batch;
  plan->D = int(D);
  plan->P = int(P);
  plan->bf16 = act == KDA_BF16;
  return KDA_OK;
}

int plan_logits(const kda_logits_args* a, kda::LogitsParams* p, bool* bf16) {
  if (a == nullptr) return fail(KDA_E_ARG, "logits arguments are NULL");
  if (a->batch < 0 || a->num_request_rows < 0 || a->max_len < 0 ||
      a->num_biases < 0 || a->num_masks < 0)
    return fail(KDA_E_ARG, "a count is negative");
  const kda_tensor& x = a->logits;
  KDA_TRY(check_desc(x, "logits", 2));
  const int64_t M = x.shape[0], V = x.shape[1];
  if (V < 1) return fail(KDA_E_SHAPE, "the logits have no vocabulary");
  if (V > (1 << 20))
    return fail(KDA_E_UNSUPPORTED, "vocabularies of up to 2^20 are supported");
  if ((V > 1 && x.stride[1] != 1) || x.stride[0] < 0)
    return fail(KDA_E_LAYOUT, "logit rows must be contiguous");
  if (M > 1 && x.stride[0] < V)
    return fail(KDA_E_LAYOUT, "logit rows overlap");
  if (!aligned(x.data, elem_size(x.dtype)))
    return fail(KDA_E_UNALIGNED, "the logits are not element aligned");
  if (!a->query_start_loc && a->batch != M)
    return fail(KDA_E_SHAPE,
                "without query_start_loc there is one request per row (%lld "
                "rows, %d requests)",
                (long long)M, a->batch);
  if (M > kI32Max - 64 || a->batch > 65535)
    return fail(KDA_E_CAPACITY, "at most 65535 requests and 2^31 rows");
  if (a->draft_tokens && !a->query_start_loc)
    return fail(KDA_E_ARG, "draft_tokens need query_start_loc");
  if (a->token_ids && a->num_request_rows > 0 &&
      (!a->prompt_lens || !a->token_lens))
    return fail(KDA_E_ARG, "token_ids need prompt_lens and token_lens");
  if (a->bias_start && a->num_biases > 0 &&
      (!a->bias_tokens || !a->bias_values))
    return fail(KDA_E_ARG, "bias_start needs bias_tokens and bias_values");
  if ((a->token_ids && a->num_request_rows > 1 &&
       a->token_ids_stride < a->max_len) ||
      (a->mask && a->num_masks > 1 && a->mask_stride < (V + 31) / 32))
    return fail(KDA_E_LAYOUT, "rows of token_ids or mask overlap");
  const void* all[] = {a->query_start_loc, a->draft_tokens,
                       a->request_indices, a->token_ids, a->prompt_lens,
                       a->token_lens, a->repetition_penalty,
                       a->frequency_penalty, a->presence_penalty,
                       a->bias_start, a->bias_tokens, a->bias_values, a->mask,
                       a->mask_rows};
  for (const void* q : all)
    if (q && !aligned(q, 4))
      return fail(KDA_E_UNALIGNED, "arrays must be 4-byte aligned");
  *p = kda::LogitsParams{};
  p->logits = x.data;
  p->s_row = x.stride[0];
  p->qsl = a->query_start_loc;
  p->draft = a->draft_tokens;
  p->req_idx = a->request_indices;
  p->tokens = a->token_ids;
  p->s_tok = a->token_ids_stride;
  p->prompt = a->prompt_lens;
  p->known = a->token_lens;
  p->rep = a->repetition_penalty;
  p->freq = a->frequency_penalty;
  p->pres = a->presence_penalty;
  p->bias_start = a->bias_start;
  p->bias_tokens = a->bias_tokens;
  p->bias_values = a->bias_values;
  p->mask = a->mask;
  p->s_mask = a->mask_stride;
  p->mask_rows = a->mask_rows;
  p->M = int32_t(M);
  p->V = int32_t(V);
  p->B = a->batch;
  p->rows = a->num_request_rows;
  p->L = a->max_len;
  p->num_bias = a->num_biases;
  p->num_masks = a->num_masks;
  *bf16 = x.dtype == KDA_BF16;
  return KDA_OK;
}

int check_pointers(std::initializer_list<const void*> needed,
                   std::initializer_list<const void*> all) {
  for (const void* q : needed)
    if (!q) return fail(KDA_E_ARG, "a required array is NULL");
  for (const void* q : all)
    if (q && !aligned(q, 4))
      return fail(KDA_E_UNALIGNED, "arrays must be 4-byte aligned");
  return KDA_OK;
}

// A block table of `rows` x `width`; one that is written must have an entry
// of its own for each element.
int check_table(const int32_t* t, const int64_t* strides, int64_t rows,
                int64_t width, bool written) {
  const int64_t sr = strides[0], sc = strides[1];
  if (rows > 0 && width > 0 && !t)
    return fail(KDA_E_ARG, "a block table is NULL");
  if (sr < 0 || sc < 0 || sr > kI32Max || sc > kI32Max)
    return fail(KDA_E_LAYOUT, "a table stride is negative or exceeds 2^31");
  if (written && width > 0 && rows > 0 &&
      ((width > 1 && sc == 0) ||
       (rows > 1 && sr < sc * (width - 1) + 1 &&
        (sr == 0 || sc < sr * (rows - 1) + 1))))
    return fail(KDA_E_LAYOUT, "the block table's rows overlap");
  return KDA_OK;
}

int plan_copy(const kda_copy_args* a, kda::CopyParams* p, int64_t* pieces) {
  if (a == nullptr) return fail(KDA_E_ARG, "copy arguments are NULL");
  if (a->num_pools < 1 || a->max_pairs < 0 || a->num_blocks < 0)
    return fail(KDA_E_ARG, "copies need a pool and no negative counts");
  if (a->null_block_id < 0)
    return fail(KDA_E_ARG, "null_block_id must not be negative");
  if (a->num_pools > 65535 || a->num_blocks > kI32Max)
    return fail(KDA_E_CAPACITY, "at most 65535 pools and 2^31 blocks");
  if (!a->tables) return fail(KDA_E_ARG, "the pools' tables are required");
  if (a->max_pairs > 0 && !a->copy_pairs)
    return fail(KDA_E_ARG, "copy_pairs is required");
  if (!aligned(a->tables, 8) || !aligned(a->copy_pairs, 4) ||
      !aligned(a->num_pairs, 4))
    return fail(KDA_E_UNALIGNED, "arrays must be aligned to their elements");
  *pieces = int64_t(1) << 20;
  if (a->host_tables) {
    const int64_t L = a->num_pools;
    int64_t most = 0;
    for (int64_t i = 0; i < L; ++i) {
      const int64_t base = a->host_tables[i], st = a->host_tables[L + i],
                    size = a->host_tables[2 * L + i];
      if (size < 1 || st < size)
        return fail(KDA_E_LAYOUT,
                    "blocks of pool %lld overlap (%lld bytes every %lld)",
                    (long long)i, (long long)size, (long long)st);
      if (base == 0) return fail(KDA_E_ARG, "a pool's address is NULL");
      most = std::max(most, kda::copy_pieces(size));
    }
    *pieces = most * std::max(a->max_pairs, 1);
  }
  *p = kda::CopyParams{a->tables,     a->copy_pairs, a->num_pairs,
                       a->num_blocks, a->num_pools,  a->max_pairs,
                       a->null_block_id};
  return KDA_OK;
}

int plan_fork(const kda_fork_args* a, kda::ForkParams* p) {
  if (a == nullptr) return fail(KDA_E_ARG, "fork arguments are NULL");
  if (a->num_forks < 0 || a->num_request_rows < 0 ||
      a->block_table_width < 0 || a->num_free < 0)
    return fail(KDA_E_ARG, "a count is negative");
  if (a->block_size < 1)
    return fail(KDA_E_ARG, "block_size must be at least 1");
  if (a->null_block_id < 0)
    return fail(KDA_E_ARG, "null_block_id must not be negative");
  if (a->num_forks > kMaxGroups)
    return fail(KDA_E_CAPACITY, "too many forks");
  if (a->num_forks > 0) {
    KDA_TRY(check_pointers({a->parent_rows, a->child_rows, a->copy_pairs,
                            a->num_allocated}, {}));
    if (a->num_request_rows > 0)
      KDA_TRY(check_pointers({a->num_computed_tokens, a->num_blocks}, {}));
    if (a->num_free > 0) KDA_TRY(check_pointers({a->free_blocks}, {}));
  }
  KDA_TRY(check_pointers({}, {a->parent_rows, a->child_rows,
                              a->num_computed_tokens, a->num_blocks,
                              a->block_table, a->free_blocks, a->copy_pairs,
                              a->num_allocated}));
  KDA_TRY(check_table(a->block_table, a->block_table_strides,
                      a->num_request_rows, a->block_table_width, true));
  *p = kda::ForkParams{a->parent_rows, a->child_rows,
                       a->num_computed_tokens, a->num_blocks, a->block_table,
                       a->block_table_strides[0], a->block_table_strides[1],
                       a->free_blocks, a->copy_pairs, a->num_allocated,
                       a->num_forks, a->num_request_rows,
                       a->block_table_width, a->block_size, a->num_free,
                       a->null_block_id};
  return KDA_OK;
}

constexpr int64_t kMaxBlocks = 1 << 28;

// Counts of chunks, then an entry a block.
int64_t blocks_bytes(int64_t N) {
  if (N < 0 || N > kMaxBlocks) return 0;
  return (N / kda::kBlockChunk + 1 + N) * 4;
}

// What the two operators over all blocks share.
template <class Args>
int check_blocks(const Args* a) {
  if (a->num_request_rows < 0 || a->block_table_width < 0 ||
      a->total_blocks < 1)
    return fail(KDA_E_ARG, "a count is negative, or there are no blocks");
  if (a->null_block_id < 0)
    return fail(KDA_E_ARG, "null_block_id must not be negative");
  if (a->total_blocks > kMaxBlocks)
    return fail(KDA_E_CAPACITY, "at most 2^28 blocks");
  if (a->num_request_rows > kMaxGroups)
    return fail(KDA_E_CAPACITY, "too many request rows");
  if (a->num_request_rows > 0)
    KDA_TRY(check_pointers({a->num_blocks}, {a->num_blocks}));
  KDA_TRY(check_table(a->block_table, a->block_table_strides,
                      a->num_request_rows, a->block_table_width, false));
  KDA_TRY(check_pointers({a->workspace}, {a->workspace, a->block_table}));
  if (a->workspace_bytes < blocks_bytes(a->total_blocks))
    return fail(KDA_E_CAPACITY,
                "the workspace holds %lld bytes; %d blocks need %lld",
                (long long)a->workspace_bytes, a->total_blocks,
                (long long)blocks_bytes(a->total_blocks));
  return KDA_OK;
}

int plan_free(const kda_free_args* a, kda::FreeParams* p) {
  if (a == nullptr) return fail(KDA_E_ARG, "free arguments are NULL");
  if (a->num_released < 0) return fail(KDA_E_ARG, "a count is negative");
  KDA_TRY(check_blocks(a));
  KDA_TRY(check_pointers({a->ref_counts, a->free_blocks, a->num_free},
                         {a->released_rows, a->pinned, a->new_num_blocks,
                          a->ref_counts, a->free_blocks, a->num_free}));
  if (a->num_released > 0) KDA_TRY(check_pointers({a->released_rows}, {}));
  if (a->num_request_rows > 0)
    KDA_TRY(check_pointers({a->new_num_blocks}, {}));
  *p = kda::FreeParams{a->released_rows, a->num_blocks, a->new_num_blocks,
                       a->block_table, a->block_table_strides[0],
                       a->block_table_strides[1], a->pinned, a->ref_counts,
                       a->free_blocks, a->num_free,
                       static_cast<int32_t*>(a->workspace), a->total_blocks,
                       a->num_released, a->num_request_rows,
                       a->block_table_width, a->null_block_id};
  return KDA_OK;
}

int plan_compact_blocks(const kda_compact_blocks_args* a,
                        kda::CompactBlocksParams* p) {
  if (a == nullptr) return fail(KDA_E_ARG, "compaction arguments are NULL");
  if (a->max_pairs < 0) return fail(KDA_E_ARG, "a count is negative");
  KDA_TRY(check_blocks(a));
  KDA_TRY(check_table(a->new_block_table, a->new_block_table_strides,
                      a->num_request_rows, a->block_table_width, true));
  KDA_TRY(check_pointers({a->ref_counts, a->new_ref_counts, a->num_pairs},
                         {a->ref_counts, a->new_ref_counts, a->num_pairs,
                          a->new_block_table, a->copy_pairs}));
  if (a->max_pairs > 0) KDA_TRY(check_pointers({a->copy_pairs}, {}));
  int32_t* work = static_cast<int32_t*>(a->workspace);
  *p = kda::CompactBlocksParams{
      a->ref_counts, a->new_ref_counts, a->num_blocks, a->block_table,
      a->block_table_strides[0], a->block_table_strides[1],
      a->new_block_table, a->new_block_table_strides[0],
      a->new_block_table_strides[1], a->copy_pairs, a->num_pairs, work,
      work + a->total_blocks / kda::kBlockChunk + 1, a->total_blocks,
      a->max_pairs, a->num_request_rows, a->block_table_width,
      a->null_block_id};
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_check_latent_write(const kda_latent_write_args* args) {
  g_err.clear();
  kda::LatentWriteParams p;
  return plan_latent_write(args, &p);
}

int kda_latent_write(const kda_latent_write_args* args, void* stream) {
  g_err.clear();
  kda::LatentWriteParams p;
  KDA_TRY(plan_latent_write(args, &p));
  if (p.T == 0) return KDA_OK;
  return device_status(
      kda::launch_latent_write(p, static_cast<hipStream_t>(stream)),
      "kda_latent_write launch");
}

int64_t kda_latent_attention_workspace_size(int64_t tokens, int64_t batch,
                                            int64_t num_heads,
                                            int64_t latent_dim,
                                            int64_t rope_dim,
                                            int32_t act_dtype) {
  if (elem_size(act_dtype) == 0) return 0;
  return latent_bytes(tokens, batch, num_heads, latent_dim, rope_dim);
}

int kda_check_latent_attention(const kda_latent_args* args) {
  g_err.clear();
  LatentPlan plan;
  return plan_latent(args, &plan);
}

int kda_latent_attention(const kda_latent_args* args, void* stream) {
  g_err.clear();
  LatentPlan plan;
  KDA_TRY(plan_latent(args, &plan));
  if (plan.noop) return KDA_OK;
  return device_status(kda::launch_latent(plan.p, plan.R, plan.P, plan.bf16,
                                          static_cast<hipStream_t>(stream)),
                       "kda_latent_attention launch");
}

int kda_check_latent_expand(const kda_latent_expand_args* args) {
  g_err.clear();
  kda::ExpandParams p{};
  bool bf16 = false;
  return plan_expand(args, &p, &bf16);
}

int kda_latent_expand(const kda_latent_expand_args* args, void* stream) {
  g_err.clear();
  kda::ExpandParams p{};
  bool bf16 = false;
  KDA_TRY(plan_expand(args, &p, &bf16));
  if (p.S == 0 || p.c.B == 0) return KDA_OK;
  return device_status(
      kda::launch_latent_expand(p, bf16, static_cast<hipStream_t>(stream)),
      "kda_latent_expand launch");
}

int kda_check_latent_prefill(const kda_latent_prefill_args* args) {
  g_err.clear();
  PromptPlan plan;
  return plan_prompt(args, &plan);
}

int kda_latent_prefill(const kda_latent_prefill_args* args, void* stream) {
  g_err.clear();
  PromptPlan plan;
  KDA_TRY(plan_prompt(args, &plan));
  if (plan.noop) return KDA_OK;
  return device_status(
      kda::launch_latent_prefill(plan.p, plan.D, plan.P, plan.bf16,
                                 static_cast<hipStream_t>(stream)),
      "kda_latent_prefill launch");
}

int kda_check_adjust_logits(const kda_logits_args* args) {
  g_err.clear();
  kda::LogitsParams p;
  bool bf16 = false;
  return plan_logits(args, &p, &bf16);
}

int kda_adjust_logits(const kda_logits_args* args, void* stream) {
  g_err.clear();
  kda::LogitsParams p;
  bool bf16 = false;
  KDA_TRY(plan_logits(args, &p, &bf16));
  if (p.M == 0 || p.B == 0) return KDA_OK;
  return device_status(
      kda::launch_adjust_logits(p, bf16, static_cast<hipStream_t>(stream)),
      "kda_adjust_logits launch");
}

int kda_check_copy_blocks(const kda_copy_args* args) {
  g_err.clear();
  kda::CopyParams p;
  int64_t pieces = 0;
  return plan_copy(args, &p, &pieces);
}

int kda_copy_blocks(const kda_copy_args* args, void* stream) {
  g_err.clear();
  kda::CopyParams p;
  int64_t pieces = 0;
  KDA_TRY(plan_copy(args, &p, &pieces));
  if (p.P == 0) return KDA_OK;
  return device_status(
      kda::launch_copy_blocks(p, pieces, static_cast<hipStream_t>(stream)),
      "kda_copy_blocks launch");
}

int kda_check_fork_blocks(const kda_fork_args* args) {
  g_err.clear();
  kda::ForkParams p;
  return plan_fork(args, &p);
}

int kda_fork_blocks(const kda_fork_args* args, void* stream) {
  g_err.clear();
  kda::ForkParams p;
  KDA_TRY(plan_fork(args, &p));
  if (p.F == 0 && !p.allocated) return KDA_OK;
  return device_status(
      kda::launch_fork_blocks(p, static_cast<hipStream_t>(stream)),
      "kda_fork_blocks launch");
}

int64_t kda_blocks_workspace_size(int64_t total_blocks) {
  return blocks_bytes(total_blocks);
}

int kda_check_free_blocks(const kda_free_args* args) {
  g_err.clear();
  kda::FreeParams p;
  return plan_free(args, &p);
}

int kda_free_blocks(const kda_free_args* args, void* stream) {
  g_err.clear();
  kda::FreeParams p;
  KDA_TRY(plan_free(args, &p));
  return device_status(
      kda::launch_free_blocks(p, static_cast<hipStream_t>(stream)),
      "kda_free_blocks launch");
}

int kda_check_compact_blocks(const kda_compact_blocks_args* args) {
  g_err.clear();
  kda::CompactBlocksParams p;
  return plan_compact_blocks(args, &p);
}

int kda_compact_blocks(const kda_compact_blocks_args* args, void* stream) {
  g_err.clear();
  kda::CompactBlocksParams p;
  KDA_TRY(plan_compact_blocks(args, &p));
  return device_status(
      kda::launch_compact_blocks(p, static_cast<hipStream_t>(stream)),
      "kda_compact_blocks launch");
}

}  // extern "C"
