// What the attention kernels (attention_*.hip) and the host side of
// kvstore_attention_paged share.  Internal to libkvstore.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kvattn __attribute__((visibility("hidden"))) {

enum Fmt { kFmt16 = 0, kFmtE4M3 = 1, kFmtE5M2 = 2, kFmtFp4 = 3 };
// Scales of an FP8 cache (the values of KVSTORE_SCALES_*).
enum ScaleKind { KVATTN_TENSOR = 0, KVATTN_TOKEN = 1, KVATTN_TOKEN_HEAD = 2 };

struct Side {   // K or V cache
  const uint8_t* data;
  int64_t page, offset, head;
  const uint8_t* scales;   // fp32 scalar, fp32 cache or e8m0 cache (see scale_kind)
  int64_t s_page, s_offset, s_head;
};

struct Params {
  const uint8_t* q;
  uint8_t* out;
  int64_t q_token, q_head, o_token, o_head;
  const int32_t* cu_q;     // NULL: sequence b is row b
  const int32_t* table;
  const int32_t* seq_lens;
  int64_t table_stride;
  Side k, v;
  float* ws_o;             // [rows, splits, dim] unnormalised sums
  float* ws_ml;            // [rows, splits, 2] maximum (log2 domain) and sum
  unsigned long long* flag;
  uint32_t tokens, seqs;
  uint32_t tile_slots;     // slots of row tiles (see tile_of)
  uint32_t kv_heads, group;   // group: q heads per kv head
  int32_t dim;
  int32_t page_size, page_shift;   // page_shift: -1 unless a power of two
  int32_t num_pages;
  int32_t max_keys;        // max_pages * page_size
  int32_t window, sinks;   // window: INT32_MAX where there is none
  float scale2;            // sm_scale * log2(e)
  int32_t scale_kind;
  int32_t chunk_steps;     // steps of a split
  int32_t splits;          // splits that the workspace has room for
  uint32_t join_parts;     // blocks of a tile in the kernel that joins splits
};

// Keys of a step and rows of a tile of the split kernel and of the tile kernel.
constexpr int kSplitStep = 32;
constexpr int kSplitRows = 16;
constexpr int kTileStep = 64;
constexpr int kTileRows = 128;

// One per (source type, format); each returns a KVSTORE_* status.
typedef int (*Launch)(const Params& p, int padded_dim, hipStream_t stream);
int launch_split_bf16_0(const Params&, int, hipStream_t);
int launch_split_bf16_1(const Params&, int, hipStream_t);
int launch_split_bf16_2(const Params&, int, hipStream_t);
int launch_split_bf16_3(const Params&, int, hipStream_t);
int launch_split_fp16_0(const Params&, int, hipStream_t);
int launch_split_fp16_1(const Params&, int, hipStream_t);
int launch_split_fp16_2(const Params&, int, hipStream_t);
int launch_split_fp16_3(const Params&, int, hipStream_t);

int launch_tile_bf16_0(const Params&, int, hipStream_t);
int launch_tile_bf16_1(const Params&, int, hipStream_t);
int launch_tile_bf16_2(const Params&, int, hipStream_t);
int launch_tile_bf16_3(const Params&, int, hipStream_t);
int launch_tile_fp16_0(const Params&, int, hipStream_t);
int launch_tile_fp16_1(const Params&, int, hipStream_t);
int launch_tile_fp16_2(const Params&, int, hipStream_t);
int launch_tile_fp16_3(const Params&, int, hipStream_t);

}  // namespace kvattn
