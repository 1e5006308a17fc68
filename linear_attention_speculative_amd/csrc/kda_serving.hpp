// Launch descriptors of the serving-step operators around the verify:
// prefill, decode, step tables and sampling.  Not part of the public ABI.
#pragma once

#include "kda_layer.hpp"

namespace kda {

struct DecodeParams {
  LayerParams y;
  const int32_t* final_slots;  // [B] or null (in place)
};
int launch_decode(const DecodeParams& p, int D, bool act_bf16,
                  hipStream_t stream);

struct PrefillParams {
  LayerParams y;
  const int32_t* qsl;        // [B + 1]
  const int32_t* initial;    // [B] or null (zeros)
  char* work;
  int32_t* order;            // [B] requests by falling length; [-1]: how many
                             // are not empty
  int32_t T;
  int32_t n_slots;           // chunk slots in the workspace
};
// Tokens per chunk, chunk slots of T tokens in B requests, and workspace
// bytes of one (chunk slot, head).
constexpr int kChunk = 32;
constexpr int64_t prefill_slots(int64_t T, int64_t B) {
  return T / kChunk + B + 1;
}
int64_t prefill_slot_bytes(int D);
int launch_prefill(const PrefillParams& p, int D, bool act_bf16,
                   hipStream_t stream);

struct TablesParams {
  const int32_t* query_lens;
  const int32_t* computed;
  const int32_t* held;
  const int32_t* req_idx;     // or null
  const int32_t* free_blocks;
  int32_t* table;
  int64_t s_tab_row, s_tab_col;
  int32_t* qsl;
  int32_t* new_held;
  int32_t* slots;
  int32_t* initial;
  int32_t* final_slots;
  int32_t* positions;
  int64_t* slot_mapping;
  int32_t* allocated;
  int32_t B, rows, width, block, num_free, cap, null_id;
};
int launch_step_tables(const TablesParams& p, hipStream_t stream);

struct SampleParams {
  const void* logits;
  int64_t s_row;
  const float* uniform;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const int32_t* qsl;         // or null
  const int32_t* draft;       // or null
  int32_t* tokens;
  int32_t* accepted;
  int32_t* next;
  char* work;
  int32_t M, V, B;
};
int64_t sample_work_bytes(int64_t M, int64_t V);
int launch_sample(const SampleParams& p, bool bf16, hipStream_t stream);

}  // namespace kda
