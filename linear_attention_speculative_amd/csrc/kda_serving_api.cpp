// Host side of the serving-step operators (prefill, decode, step tables,
// sampling): argument checks, translation of the public descriptors into
// launch parameters, and the exported C entry points.
#include <stdint.h>

#include <algorithm>

#include "kda_host.hpp"
#include "kda_recoverssm.h"
#include "kda_serving.hpp"

using namespace kda::host;

namespace {

constexpr int64_t kI32Max = 0x7fffffff;
constexpr int64_t kMaxThreads = 0xffffffff;   // work items of a launch

// The fields that the two layer argument blocks share.
struct LayerView {
  const kda_tensor &mixed_qkv, &raw_gate, &raw_beta, &A_log, &dt_bias, &state,
      &out, &conv_state, &conv_weight;
  int32_t batch, Q, null_id, dim_first, use_lb;
  float lb;
  const int32_t* slots;
  const int32_t* accepted;
};

template <class Args>
LayerView view_of(const Args* a) {
  return LayerView{a->mixed_qkv,      a->raw_gate,        a->raw_beta,
                   a->A_log,          a->dt_bias,         a->state,
                   a->out,            a->conv_state,      a->conv_weight,
                   a->batch,          a->spec_query_len,  a->null_block_id,
                   a->conv_dim_first, a->use_lower_bound, a->lower_bound,
                   a->state_indices,  a->num_accepted_tokens};
}

// Whether a tensor of three dimensions has its elements in places of their own,
// each dimension's stride past the extent of those of smaller stride.
bool nested(const kda_tensor& t) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3,
            [&](int i, int j) { return t.stride[i] < t.stride[j]; });
  int64_t extent = 0;          // from the first element to the last
  for (int i : order) {
    if (t.shape[i] <= 1) continue;
    if (t.stride[i] <= extent) return false;
    extent += (t.shape[i] - 1) * t.stride[i];
  }
  return true;
}

// Checks of one layer's tensors (the verify's rules where they apply), and
// their translation.
int plan_layer(const LayerView& a, bool conv, kda::LayerParams* p, int* D_out,
               bool* act_bf16, int64_t* T_out) {
  if (a.batch < 0) return fail(KDA_E_ARG, "batch is negative");
  KDA_TRY(check_desc(a.A_log, "A_log", 1));
  KDA_TRY(check_desc(a.state, "state", 4));
  const kda_tensor& S = a.state;
  const int64_t H = a.A_log.shape[0], N = S.shape[0], D = S.shape[3];
  if (H < 1) return fail(KDA_E_SHAPE, "A_log must hold one value per head");
  if (S.dtype != KDA_F32)
    return fail(KDA_E_DTYPE, "the state must be float32");
  if (!supported_head_dim(D))
    return fail(KDA_E_UNSUPPORTED,
                "head dim %lld is not supported (16, 32, 64 or 128)",
                (long long)D);
  if (N < 1 || S.shape[1] != H || S.shape[2] != D)
    return fail(KDA_E_SHAPE,
                "state must be [slots, heads=%lld, %lld, %lld]", (long long)H,
                (long long)D, (long long)D);
  if (S.stride[1] != D * D || S.stride[2] != D || S.stride[3] != 1 ||
      S.stride[0] < 0 || (S.stride[0] * 4) % 16 != 0)
    return fail(KDA_E_LAYOUT,
                "the state needs contiguous heads and 16-byte aligned slots");
  if (a.A_log.dtype != KDA_F32)
    return fail(KDA_E_DTYPE, "A_log must be float32");
  if (H > 1 && a.A_log.stride[0] != 1)
    return fail(KDA_E_LAYOUT, "A_log must be contiguous");
  const kda_tensor& dtb = a.dt_bias;
  if (dtb.ndim != 1 && dtb.ndim != 2)
    return fail(KDA_E_SHAPE, "dt_bias must be [H*D] or [H, D]");
  KDA_TRY(check_desc(dtb, "dt_bias", dtb.ndim));
  if (dtb.dtype != KDA_F32)
    return fail(KDA_E_DTYPE, "dt_bias must be float32");
  if (dtb.ndim == 1 ? (dtb.shape[0] != H * D || dtb.stride[0] != 1)
                    : (dtb.shape[0] != H || dtb.shape[1] != D ||
                       dtb.stride[1] != 1 || dtb.stride[0] != D))
    return fail(KDA_E_SHAPE,
                "dt_bias must hold heads*head_dim contiguous values");

  KDA_TRY(check_desc(a.mixed_qkv, "mixed_qkv", 2));
  KDA_TRY(check_desc(a.raw_gate, "raw_gate", 2));
  KDA_TRY(check_desc(a.raw_beta, "raw_beta", 2));
  KDA_TRY(check_desc(a.out, "out", 2));
  const int32_t act = a.mixed_qkv.dtype;
  const int64_t T = a.mixed_qkv.shape[0], HD = H * D;
  if (a.raw_gate.dtype != act || a.raw_beta.dtype != act)
    return fail(KDA_E_DTYPE,
                "mixed_qkv, raw_gate and raw_beta must share one dtype");
  if (a.out.dtype != KDA_F32 && a.out.dtype != act)
    return fail(KDA_E_DTYPE, "out must be float32 or the activation dtype");
  if (!shape_is(a.mixed_qkv, T, 3 * HD))
    return fail(KDA_E_SHAPE, "mixed_qkv must be [T, 3*H*D] = [%lld, %lld]",
                (long long)T, (long long)(3 * HD));
  if (!shape_is(a.raw_gate, T, HD) || !shape_is(a.raw_beta, T, H) ||
      !shape_is(a.out, T, HD))
    return fail(KDA_E_SHAPE,
                "raw_gate, raw_beta and out must be [T, H*D], [T, H] and "
                "[T, H*D] with the T = %lld rows of mixed_qkv",
                (long long)T);
  if (a.mixed_qkv.stride[1] != 1 || a.raw_gate.stride[1] != 1 ||
      (H > 1 && a.raw_beta.stride[1] != 1) || a.out.stride[1] != 1)
    return fail(KDA_E_LAYOUT,
                "activation and output rows must be contiguous");

  const kda_tensor none{};
  const kda_tensor& cs = conv ? a.conv_state : none;
  const kda_tensor& cw = conv ? a.conv_weight : none;
  int64_t s_chan = 0, s_tok = 0;
  if (conv) {
    if (a.Q < 1 || a.Q > kda::kMaxWindow)
      return fail(KDA_E_UNSUPPORTED,
                  "draft windows of 1 to %d positions are supported (got %d)",
                  kda::kMaxWindow, a.Q);
    KDA_TRY(check_desc(cs, "conv_state", 3));
    KDA_TRY(check_desc(cw, "conv_weight", 2));
    const int64_t C = a.dim_first ? cs.shape[1] : cs.shape[2];
    const int64_t Lc = a.dim_first ? cs.shape[2] : cs.shape[1];
    s_chan = a.dim_first ? cs.stride[1] : cs.stride[2];
    s_tok = a.dim_first ? cs.stride[2] : cs.stride[1];
    if (cs.shape[0] != N || C != 3 * HD)
      return fail(KDA_E_SHAPE,
                  "conv state must be [slots=%lld, %lld, Lc] (dim first) or "
                  "[slots, Lc, %lld] (token first)",
                  (long long)N, (long long)(3 * HD), (long long)(3 * HD));
    if (cs.dtype != act)
      return fail(KDA_E_DTYPE,
                  "the conv state must use the activation dtype (%s)",
                  dt_name(act));
    if (Lc != a.Q + kda::kConvWidth - 2)
      return fail(KDA_E_UNSUPPORTED,
                  "conv state length %lld does not fit a width-%d "
                  "convolution (length = Q + 2 = %d)",
                  (long long)Lc, kda::kConvWidth, a.Q + 2);
    if (!shape_is(cw, 3 * HD, kda::kConvWidth))
      return fail(KDA_E_SHAPE, "conv_weight must be [%lld, %d]",
                  (long long)(3 * HD), kda::kConvWidth);
    if (cw.dtype != KDA_F32 && cw.dtype != act)
      return fail(KDA_E_DTYPE,
                  "conv_weight must be float32 or the activation dtype");
  }
  if (int64_t(a.batch) * H > kI32Max || T > kI32Max || N > kI32Max)
    return fail(KDA_E_CAPACITY, "batch * heads, tokens or slots exceed 2^31");

  const kda_tensor* statics[] = {&a.state, &a.A_log, &a.dt_bias, &cs, &cw};
  const char* names[] = {"state", "A_log", "dt_bias", "conv_state",
                         "conv_weight"};
  for (int i = 0; i < 5; ++i)
    if (!aligned(statics[i]->data, 16))
      return fail(KDA_E_LAYOUT, "%s must start on a 16-byte boundary",
                  names[i]);
  const int ea = elem_size(act), eo = elem_size(a.out.dtype);
  if (!aligned(a.mixed_qkv.data, 16) || !aligned(a.raw_gate.data, 16) ||
      !aligned(a.out.data, 16) || (a.mixed_qkv.stride[0] * ea) % 16 != 0 ||
      (a.raw_gate.stride[0] * ea) % 16 != 0 ||
      (a.out.stride[0] * eo) % 16 != 0)
    return fail(KDA_E_UNALIGNED,
                "an activation or output row does not start on a 16-byte "
                "boundary");
  if (!aligned(a.raw_beta.data, ea))
    return fail(KDA_E_UNALIGNED, "raw_beta is not element aligned");
  const int64_t strides[] = {a.mixed_qkv.stride[0], a.raw_gate.stride[0],
                             a.raw_beta.stride[0],  a.out.stride[0],
                             cs.stride[0],          cs.stride[1],
                             cs.stride[2],          cw.stride[0],
                             cw.stride[1]};
  for (int64_t st : strides)
    if (st < 0 || st > kI32Max)
      return fail(KDA_E_LAYOUT, "a tensor stride is negative or exceeds 2^31");
  // Elements that writes would share (a broadcast or sliding view) cannot hold
  // results.
  if (conv && !nested(cs))
    return fail(KDA_E_LAYOUT, "the conv state's entries overlap");
  if (T > 1 && a.out.stride[0] < HD)
    return fail(KDA_E_LAYOUT, "out's rows overlap");
  if (N > 1 && S.stride[0] < H * D * D)
    return fail(KDA_E_LAYOUT, "the state's slots overlap");
  if (a.batch > 0) {
    if (!a.slots) return fail(KDA_E_ARG, "state_indices is required");
    if (!aligned(a.slots, 4) || (a.accepted && !aligned(a.accepted, 4)))
      return fail(KDA_E_UNALIGNED, "metadata pointers must be 4-byte aligned");
  }

  *p = kda::LayerParams{};
  p->mixed_qkv = a.mixed_qkv.data;
  p->raw_gate = a.raw_gate.data;
  p->raw_beta = a.raw_beta.data;
  p->A_log = static_cast<const float*>(a.A_log.data);
  p->dt_bias = static_cast<const float*>(dtb.data);
  p->state = static_cast<float*>(S.data);
  p->out = a.out.data;
  p->conv_state = cs.data;
  p->conv_weight = cw.data;
  p->s_x = a.mixed_qkv.stride[0];
  p->s_g = a.raw_gate.stride[0];
  p->s_beta = a.raw_beta.stride[0];
  p->s_out = a.out.stride[0];
  p->s_slot = S.stride[0];
  p->s_cs_slot = cs.stride[0];
  p->s_cs_chan = s_chan;
  p->s_cs_tok = s_tok;
  p->s_w_chan = cw.stride[0];
  p->s_w_tap = cw.stride[1];
  p->slots = a.slots;
  p->accepted = conv ? a.accepted : nullptr;
  p->B = a.batch;
  p->H = int32_t(H);
  p->N = int32_t(N);
  p->Q = a.Q;
  p->null_id = a.null_id;
  p->flags = (a.out.dtype == KDA_BF16 ? kda::kOutBf16 : 0) |
             (conv && cw.dtype == KDA_BF16 ? kda::kWBf16 : 0) |
             (conv ? 0 : kda::kNoConv) | (a.use_lb ? kda::kLowerBound : 0);
  // each channel's four taps contiguous and aligned to their size
  if (conv && cw.stride[1] == 1 && cw.stride[0] == kda::kConvWidth &&
      aligned(cw.data, uintptr_t(kda::kConvWidth) * elem_size(cw.dtype)))
    p->flags |= kda::kWRow;
  p->lb = a.lb;
  *D_out = int(D);
  *act_bf16 = act == KDA_BF16;
  *T_out = T;
  return KDA_OK;
}

struct PrefillPlan {
  kda::PrefillParams p;
  int D = 0;
  bool act_bf16 = false;
  bool noop = false;
};

// Bytes of workspace, or 0 for sizes that no launch takes.
int64_t prefill_bytes(int64_t T, int64_t B, int64_t H, int64_t D) {
  if (T < 0 || B < 0 || H < 1 || !supported_head_dim(D) || T > kI32Max ||
      B > kI32Max || H > kI32Max || B * H > kI32Max)
    return 0;
  const int64_t slots = kda::prefill_slots(T, B);
  // launches of up to 512 threads per (chunk slot, head), and of up to 320
  // per (request, head, 16 rows)
  if (slots > kMaxThreads / 512 / H ||
      (B * H + 7) / 8 * 8 * (D / 16) > kMaxThreads / 320)
    return 0;
  return slots * H * kda::prefill_slot_bytes(int(D)) +
         (B + 4) / 4 * 16;     // the order of the requests, behind the slots
}

int plan_prefill(const kda_prefill_args* a, bool conv, PrefillPlan* plan) {
  if (a == nullptr) return fail(KDA_E_ARG, "prefill arguments are NULL");
  kda::PrefillParams& p = plan->p;
  int64_t T = 0;
  KDA_TRY(plan_layer(view_of(a), conv, &p.y, &plan->D, &plan->act_bf16, &T));
  // The chunked form's operands are products of decays of at most 1 each.
  if (a->use_lower_bound && !(a->lower_bound <= 0.0f))
    return fail(KDA_E_UNSUPPORTED,
                "the prefill needs a lower_bound of at most 0 (got %g)",
                double(a->lower_bound));
  plan->noop = a->batch == 0 || T == 0;
  const int64_t need = prefill_bytes(T, a->batch, p.y.H, plan->D);
  if (need == 0)
    return fail(KDA_E_CAPACITY, "tokens, requests and heads exceed the grid");
  if (!plan->noop) {
    if (!a->query_start_loc)
      return fail(KDA_E_ARG, "query_start_loc is required");
    if (!a->workspace) return fail(KDA_E_ARG, "the workspace is required");
    if (a->workspace_bytes < need)
      return fail(KDA_E_CAPACITY,
                  "the workspace holds %lld bytes; %lld tokens of %d requests "
                  "need %lld",
                  (long long)a->workspace_bytes, (long long)T, a->batch,
                  (long long)need);
    if (!aligned(a->workspace, 16))
      return fail(KDA_E_UNALIGNED, "the workspace must be 16-byte aligned");
    if (!aligned(a->query_start_loc, 4) ||
        (a->initial_state_indices && !aligned(a->initial_state_indices, 4)))
      return fail(KDA_E_UNALIGNED, "metadata pointers must be 4-byte aligned");
  }
  p.qsl = a->query_start_loc;
  p.initial = a->initial_state_indices;
  p.work = static_cast<char*>(a->workspace);
  p.T = int32_t(T);
  p.n_slots = int32_t(kda::prefill_slots(T, a->batch));
  p.order = reinterpret_cast<int32_t*>(
                p.work + need - (int64_t(a->batch) + 4) / 4 * 16) + 1;
  return KDA_OK;
}

int run_prefill(const kda_prefill_args* a, bool conv, void* stream,
                const char* what) {
  g_err.clear();
  PrefillPlan plan;
  KDA_TRY(plan_prefill(a, conv, &plan));
  if (plan.noop) return KDA_OK;
  return device_status(
      kda::launch_prefill(plan.p, plan.D, plan.act_bf16,
                          static_cast<hipStream_t>(stream)),
      what);
}

struct DecodePlan {
  kda::DecodeParams p;
  int D = 0;
  bool act_bf16 = false;
};

int plan_decode(const kda_decode_args* a, bool conv, DecodePlan* plan) {
  if (a == nullptr) return fail(KDA_E_ARG, "decode arguments are NULL");
  int64_t T = 0;
  KDA_TRY(plan_layer(view_of(a), conv, &plan->p.y, &plan->D, &plan->act_bf16,
                     &T));
  if (T != a->batch)
    return fail(KDA_E_SHAPE,
                "a decode step takes one row per request (%lld rows, %d "
                "requests)",
                (long long)T, a->batch);
  // up to 512 threads per (request, head)
  if (T * plan->p.y.H > kMaxThreads / 512)
    return fail(KDA_E_CAPACITY, "requests and heads exceed the grid");
  if (a->final_state_indices && !aligned(a->final_state_indices, 4))
    return fail(KDA_E_UNALIGNED, "metadata pointers must be 4-byte aligned");
  plan->p.final_slots = a->final_state_indices;
  return KDA_OK;
}

int run_decode(const kda_decode_args* a, bool conv, void* stream,
               const char* what) {
  g_err.clear();
  DecodePlan plan;
  KDA_TRY(plan_decode(a, conv, &plan));
  if (plan.p.y.B == 0) return KDA_OK;
  return device_status(
      kda::launch_decode(plan.p, plan.D, plan.act_bf16,
                         static_cast<hipStream_t>(stream)),
      what);
}

int plan_tables(const kda_tables_args* a, kda::TablesParams* p) {
  if (a == nullptr) return fail(KDA_E_ARG, "step table arguments are NULL");
  if (a->batch < 0 || a->num_request_rows < 0 || a->block_table_width < 0 ||
      a->num_free < 0 || a->max_tokens < 0)
    return fail(KDA_E_ARG, "a count is negative");
  if (a->block_size < 1)
    return fail(KDA_E_ARG, "block_size must be at least 1");
  if (a->null_block_id < 0)
    return fail(KDA_E_ARG, "null_block_id must not be negative");
  const bool rows = a->num_request_rows > 0;
  const void* need[] = {a->query_start_loc, a->num_allocated};
  const void* need_b[] = {a->query_lens, a->state_indices,
                          a->initial_state_indices, a->final_state_indices};
  const void* need_r[] = {a->num_computed_tokens, a->num_blocks,
                          a->new_num_blocks};
  const void* need_t[] = {a->positions, a->slot_mapping};
  bool missing = false;
  for (const void* q : need) missing |= q == nullptr;
  if (a->batch > 0)
    for (const void* q : need_b) missing |= q == nullptr;
  if (a->batch > 0 && rows)
    for (const void* q : need_r) missing |= q == nullptr;
  if (a->max_tokens > 0)
    for (const void* q : need_t) missing |= q == nullptr;
  if (a->num_free > 0) missing |= a->free_blocks == nullptr;
  if (rows && a->block_table_width > 0) missing |= a->block_table == nullptr;
  if (missing) return fail(KDA_E_ARG, "a required array is NULL");
  const void* all[] = {a->query_lens,      a->num_computed_tokens,
                       a->num_blocks,      a->request_indices,
                       a->free_blocks,     a->block_table,
                       a->query_start_loc, a->new_num_blocks,
                       a->state_indices,   a->initial_state_indices,
                       a->final_state_indices, a->positions,
                       a->num_allocated};
  for (const void* q : all)
    if (q && !aligned(q, 4))
      return fail(KDA_E_UNALIGNED, "arrays must be 4-byte aligned");
  if (a->slot_mapping && !aligned(a->slot_mapping, 8))
    return fail(KDA_E_UNALIGNED, "slot_mapping must be 8-byte aligned");
  const int64_t sr = a->block_table_strides[0], sc = a->block_table_strides[1];
  if (sr < 0 || sc < 0 || sr > kI32Max || sc > kI32Max)
    return fail(KDA_E_LAYOUT, "a table stride is negative or exceeds 2^31");
  const int64_t width = a->block_table_width, nrows = a->num_request_rows;
  if (width > 0 && nrows > 0 &&
      ((width > 1 && sc == 0) ||
       (nrows > 1 && sr < sc * (width - 1) + 1 &&
        (sr == 0 || sc < sr * (nrows - 1) + 1))))
    return fail(KDA_E_LAYOUT, "the block table's rows overlap");
  *p = kda::TablesParams{};
  p->query_lens = a->query_lens;
  p->computed = a->num_computed_tokens;
  p->held = a->num_blocks;
  p->req_idx = a->request_indices;
  p->free_blocks = a->free_blocks;
  p->table = a->block_table;
  p->s_tab_row = sr;
  p->s_tab_col = sc;
  p->qsl = a->query_start_loc;
  p->new_held = a->new_num_blocks;
  p->slots = a->state_indices;
  p->initial = a->initial_state_indices;
  p->final_slots = a->final_state_indices;
  p->positions = a->positions;
  p->slot_mapping = a->slot_mapping;
  p->allocated = a->num_allocated;
  p->B = a->batch;
  p->rows = a->num_request_rows;
  p->width = a->block_table_width;
  p->block = a->block_size;
  p->num_free = a->num_free;
  p->cap = a->max_tokens;
  p->null_id = a->null_block_id;
  return KDA_OK;
}

int plan_sample(const kda_sample_args* a, kda::SampleParams* p, bool* bf16) {
  if (a == nullptr) return fail(KDA_E_ARG, "sampling arguments are NULL");
  if (a->batch < 0) return fail(KDA_E_ARG, "batch is negative");
  const kda_tensor& x = a->logits;
  KDA_TRY(check_desc(x, "logits", 2));
  const int64_t M = x.shape[0], V = x.shape[1];
  if (V < 1) return fail(KDA_E_SHAPE, "the logits have no vocabulary");
  if (V > (1 << 20))
    return fail(KDA_E_UNSUPPORTED, "vocabularies of up to 2^20 are supported");
  const int64_t need = kda::sample_work_bytes(M, V);
  if (need == 0) return fail(KDA_E_CAPACITY, "too many rows");
  if ((V > 1 && x.stride[1] != 1) || x.stride[0] < 0)
    return fail(KDA_E_LAYOUT, "logit rows must be contiguous");
  if (!aligned(x.data, elem_size(x.dtype)))
    return fail(KDA_E_UNALIGNED, "the logits are not element aligned");
  if (!a->query_start_loc && a->batch != M)
    return fail(KDA_E_SHAPE,
                "without query_start_loc there is one request per row (%lld "
                "rows, %d requests)",
                (long long)M, a->batch);
  if (a->draft_tokens) {
    if (!a->query_start_loc)
      return fail(KDA_E_ARG, "draft_tokens need query_start_loc");
    if (a->batch > 0 && (!a->num_accepted || !a->next_tokens))
      return fail(KDA_E_ARG,
                  "draft_tokens need num_accepted and next_tokens");
  } else if (a->num_accepted || a->next_tokens) {
    return fail(KDA_E_ARG,
                "num_accepted and next_tokens need draft_tokens");
  }
  if (M > 0) {
    if (!a->uniform || !a->tokens)
      return fail(KDA_E_ARG, "uniform and tokens are required");
    if (!a->workspace) return fail(KDA_E_ARG, "the workspace is required");
    if (a->workspace_bytes < need)
      return fail(KDA_E_CAPACITY,
                  "the workspace holds %lld bytes; %lld rows of %lld logits "
                  "need %lld",
                  (long long)a->workspace_bytes, (long long)M, (long long)V,
                  (long long)need);
    if (!aligned(a->workspace, 16))
      return fail(KDA_E_UNALIGNED, "the workspace must be 16-byte aligned");
  }
  const void* all[] = {a->uniform, a->temperature, a->top_k, a->top_p,
                       a->min_p, a->query_start_loc, a->draft_tokens,
                       a->tokens, a->num_accepted, a->next_tokens};
  for (const void* q : all)
    if (q && !aligned(q, 4))
      return fail(KDA_E_UNALIGNED, "arrays must be 4-byte aligned");
  *p = kda::SampleParams{};
  p->logits = x.data;
  p->s_row = x.stride[0];
  p->uniform = a->uniform;
  p->temperature = a->temperature;
  p->top_k = a->top_k;
  p->top_p = a->top_p;
  p->min_p = a->min_p;
  p->qsl = a->query_start_loc;
  p->draft = a->draft_tokens;
  p->tokens = a->tokens;
  p->accepted = a->num_accepted;
  p->next = a->next_tokens;
  p->work = static_cast<char*>(a->workspace);
  p->M = int32_t(M);
  p->V = int32_t(V);
  p->B = a->batch;
  *bf16 = x.dtype == KDA_BF16;
  return KDA_OK;
}

}  // namespace

extern "C" {

int64_t kda_prefill_workspace_size(int64_t tokens, int64_t batch,
                                   int64_t num_heads, int64_t head_dim,
                                   int32_t act_dtype, int32_t out_dtype) {
  if (elem_size(act_dtype) == 0 ||
      (out_dtype != KDA_F32 && out_dtype != act_dtype))
    return 0;
  return prefill_bytes(tokens, batch, num_heads, head_dim);
}

int kda_check_prefill(const kda_prefill_args* args) {
  g_err.clear();
  PrefillPlan plan;
  return plan_prefill(args, true, &plan);
}

int kda_conv_prefill(const kda_prefill_args* args, void* stream) {
  return run_prefill(args, true, stream, "kda_conv_prefill launch");
}

int kda_check_prefill_qkv(const kda_prefill_args* args) {
  g_err.clear();
  PrefillPlan plan;
  return plan_prefill(args, false, &plan);
}

int kda_prefill_qkv(const kda_prefill_args* args, void* stream) {
  return run_prefill(args, false, stream, "kda_prefill_qkv launch");
}

int kda_check_decode(const kda_decode_args* args) {
  g_err.clear();
  DecodePlan plan;
  return plan_decode(args, true, &plan);
}

int kda_conv_update_decode(const kda_decode_args* args, void* stream) {
  return run_decode(args, true, stream, "kda_conv_update_decode launch");
}

int kda_check_decode_qkv(const kda_decode_args* args) {
  g_err.clear();
  DecodePlan plan;
  return plan_decode(args, false, &plan);
}

int kda_decode_qkv(const kda_decode_args* args, void* stream) {
  return run_decode(args, false, stream, "kda_decode_qkv launch");
}

int kda_check_step_tables(const kda_tables_args* args) {
  g_err.clear();
  kda::TablesParams p;
  return plan_tables(args, &p);
}

int kda_step_tables(const kda_tables_args* args, void* stream) {
  g_err.clear();
  kda::TablesParams p;
  KDA_TRY(plan_tables(args, &p));
  return device_status(
      kda::launch_step_tables(p, static_cast<hipStream_t>(stream)),
      "kda_step_tables launch");
}

int64_t kda_sample_workspace_size(int64_t rows, int64_t vocab) {
  return kda::sample_work_bytes(rows, vocab);
}

int kda_check_sample(const kda_sample_args* args) {
  g_err.clear();
  kda::SampleParams p;
  bool bf16 = false;
  return plan_sample(args, &p, &bf16);
}

int kda_sample(const kda_sample_args* args, void* stream) {
  g_err.clear();
  kda::SampleParams p;
  bool bf16 = false;
  KDA_TRY(plan_sample(args, &p, &bf16));
  return device_status(
      kda::launch_sample(p, bf16, static_cast<hipStream_t>(stream)),
      "kda_sample launch");
}

}  // extern "C"
