// Launch descriptors of the operators on token caches, blocks and logits
// (latent attention, block life, changes of logits).  Not part of the public
// ABI.
#pragma once

#include "kda_internal.hpp"

namespace kda {

// Where a request's tokens lie: offsets, computed tokens, block table.
struct PagedParams {
  const int32_t* qsl;        // [B + 1]
  const int32_t* computed;   // per request row
  const int32_t* req_idx;    // [B] or null (row = b)
  const int32_t* table;      // [rows, width]
  int64_t s_tab_row, s_tab_col;
  const char* cache;
  int64_t s_blk, s_tok;      // bytes
  int32_t B, rows, width, block, null_id;
  int64_t N;                 // blocks of the cache
  uint32_t magic;            // position / block = position * magic >> shift,
  int32_t shift;             // for positions below 2^31
};

struct LatentWriteParams {
  const char* latent;
  const char* rope;          // or null
  int64_t s_lat, s_rope;     // bytes
  char* cache;
  int64_t s_blk, s_tok;      // bytes
  const int64_t* slots;
  int64_t total_slots;       // N * block
  int64_t first_slot;        // (slots below it are null)
  int32_t T, block;
  int32_t lat_chunks, chunks;    // 16-byte chunks of the latent, of a row
};
int launch_latent_write(const LatentWriteParams& p, hipStream_t stream);

struct LatentParams {
  PagedParams c;
  const char* q;
  int64_t s_q_tok, s_q_head;     // bytes
  char* out;
  int64_t s_out_tok, s_out_head; // bytes
  float* lse;                    // or null
  int64_t s_lse_tok, s_lse_head;
  char* work;
  float scale;                   // softmax scale times log2 e, above 0,
  int32_t negate;                // and whether that is of negated queries
  int32_t T, H;
  int32_t group;                 // rows of a workgroup / 32: 1 or 2
  int32_t workers;
};
// Row groups for these sizes, and workspace bytes.
constexpr int kLatentWorkers = 256;
int latent_groups(int64_t T, int64_t B, int64_t H);
int latent_workers(int64_t T, int64_t B, int64_t H, int64_t tokens, int group);
int64_t latent_work_bytes(int group, int R);
int launch_latent(const LatentParams& p, int R, int P, bool bf16,
                  hipStream_t stream);

struct ExpandParams {
  PagedParams c;                 // qsl: the key rows' offsets; no lengths
  const char* w;                 // [H, 2 D, R]
  int64_t s_w_head, s_w_row;     // bytes, from here on
  char* key;
  int64_t s_k_tok, s_k_head;
  char* value;
  int64_t s_v_tok, s_v_head;
  char* rope;                    // or null
  int64_t s_rope;
  int32_t S, H, D, R;
  int32_t rope_chunks;           // of 16 bytes
};
int launch_latent_expand(const ExpandParams& p, bool bf16,
                         hipStream_t stream);

struct PromptParams {
  const char* q;
  int64_t s_q_tok, s_q_head;     // bytes
  const char* key;
  int64_t s_k_tok, s_k_head;
  const char* value;
  int64_t s_v_tok, s_v_head;
  const char* rope;
  int64_t s_rope;
  char* out;
  int64_t s_out_tok, s_out_head;
  float* lse;                    // or null
  int64_t s_lse_tok, s_lse_head;
  const int32_t* qsl;
  const int32_t* ksl;
  float scale;                   // as in LatentParams
  int32_t negate;
  int32_t T, S, H, B;
};
int64_t prompt_tiles(int64_t T, int64_t B);
int launch_latent_prefill(const PromptParams& p, int D, int P, bool bf16,
                          hipStream_t stream);

struct LogitsParams {
  void* logits;
  int64_t s_row;
  const int32_t* qsl;            // or null: a row a request
  const int32_t* draft;          // or null
  const int32_t* req_idx;        // or null
  const int32_t* tokens;         // [rows, L], or null: no history
  int64_t s_tok;
  const int32_t* prompt;
  const int32_t* known;
  const float* rep;              // [B] each, or null
  const float* freq;
  const float* pres;
  const int32_t* bias_start;     // [B + 1], or null: no biases
  const int32_t* bias_tokens;
  const float* bias_values;
  const int32_t* mask;           // or null
  int64_t s_mask;
  const int32_t* mask_rows;      // [M], or null: row m
  int32_t M, V, B, rows, L, num_bias, num_masks;
  int32_t mask_from;             // first row of a launch of the masks
  int32_t parts;                 // workgroups that share a request's window
};
int launch_adjust_logits(const LogitsParams& p, bool bf16,
                         hipStream_t stream);

struct CopyParams {
  const int64_t* tables;         // [3][L]: bases, block strides and block
                                 // sizes, in bytes
  const int32_t* pairs;          // [P][2]: source, destination
  const int32_t* num_pairs;      // [1] or null: P
  int64_t N;
  int32_t L, P, null_id;
};
int64_t copy_pieces(int64_t bytes);
int launch_copy_blocks(const CopyParams& p, int64_t pieces,
                       hipStream_t stream);

struct ForkParams {
  const int32_t* parents;        // [F]
  const int32_t* children;
  int32_t* computed;             // per request row
  int32_t* held;
  int32_t* table;
  int64_t s_tab_row, s_tab_col;
  const int32_t* free_blocks;
  int32_t* pairs;                // [F][2]
  int32_t* allocated;            // [1]
  int32_t F, rows, width, block, num_free, null_id;
};
int launch_fork_blocks(const ForkParams& p, hipStream_t stream);

constexpr int kBlockChunk = 4096;   // blocks of one count
struct FreeParams {
  const int32_t* released;       // [R]
  const int32_t* held;           // per request row
  int32_t* new_held;
  const int32_t* table;
  int64_t s_tab_row, s_tab_col;
  const int32_t* pinned;         // [N] or null
  int32_t* refs;                 // [N]
  int32_t* free_blocks;          // [N]
  int32_t* num_free;             // [1]
  int32_t* counts;               // workspace: one a chunk of blocks
  int64_t N;
  int32_t R, rows, width, null_id;
};
int launch_free_blocks(const FreeParams& p, hipStream_t stream);

struct CompactBlocksParams {
  const int32_t* refs;           // [N]
  int32_t* new_refs;
  const int32_t* held;
  const int32_t* table;
  int64_t s_tab_row, s_tab_col;
  int32_t* new_table;
  int64_t s_new_row, s_new_col;
  int32_t* pairs;                // [max_pairs][2]
  int32_t* num_pairs;            // [1]
  int32_t* counts;               // workspace
  int32_t* moved;                // workspace [N]: a moved block's pair
  int64_t N;
  int32_t max_pairs, rows, width, null_id;
};
int launch_compact_blocks(const CompactBlocksParams& p, hipStream_t stream);

}  // namespace kda
