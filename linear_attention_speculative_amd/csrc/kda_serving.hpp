// Launch descriptors of the serving-step operators around the verify:
// decode and step tables.  Not part of the public ABI.
#pragma once

#include "kda_layer.hpp"

namespace kda {

struct DecodeParams {
  LayerParams y;
  const int32_t* final_slots;  // [B] or null (in place)
};
int launch_decode(const DecodeParams& p, int D, bool act_bf16,
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

}  // namespace kda
