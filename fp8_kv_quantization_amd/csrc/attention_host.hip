// Host side of kvstore_attention_paged: checks, the choice of tiles and splits,
// and dispatch.  Part of the translation unit of libkvstore.hip.

#include "attention.h"

namespace {

// The error flag's address on the current device, NULL on a runtime error
// (cached per device; calls from several threads may fill an entry
// concurrently with the same value).
unsigned long long* error_flag() {
  static std::atomic<unsigned long long*> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return nullptr;
  unsigned long long* at = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : nullptr;
  if (at != nullptr) return at;
  if (hipGetSymbolAddress(reinterpret_cast<void**>(&at), HIP_SYMBOL(g_kvstore_error)) != hipSuccess)
    return nullptr;
  if (dev < 64) cache[dev].store(at, std::memory_order_relaxed);
  return at;
}

struct AttentionPlan {
  bool split;           // the split kernel (else the tile kernel)
  int padded_dim;
  uint32_t tile_slots;
  int32_t max_keys;
  int32_t chunk_steps;
  int32_t splits;
  int64_t workspace;    // bytes
  uint32_t join_parts;  // blocks of a tile in the kernel that joins splits
};

// Up to 16 rows take the split kernel, which gets most out of few of them; more
// take the tile kernel, which reads the cache once for up to 128 (32 rows, 8
// sequences of 8192 keys, 8 kv heads of 128 dims: 54 us against the split
// kernel's 110 in two passes over 16 bits, 61 against 94 over e4m3fn, 50 against
// 56 over 4 bits).  16-bit rows of more than 64 dims go faster through the tile
// kernel's loads into LDS, however few rows there are, once there is more to read
// than kAttnTileBytes (one row of 4 heads a kv head, 8 kv heads of 128 dims: 8
// sequences of 8192 keys 50 us against 70, 16 of 1024 21.0 against 23.4, one of
// 8192 17.4 against 17.3, 4 of 2048 16 against 14.3, one of 777 14.8 against 10.8;
// of 64 dims, 8 of 8192 34.3 against 33.9; e4m3fn, 8 of 8192: 58 against 47).
constexpr int64_t kAttnTileBytes = int64_t(48) << 20;
// Blocks to aim for by splits.  Split kernel: three or four a CU run at once, and
// several turns of them even out sequences of different lengths (32 contexts of up
// to 32768 4-bit keys: 167 us with 2048, 157 with 4096, 156 with 8192; 64 windows
// of 4096: 106, 106, 109).  Tile kernel: the two a CU that run at once (single
// rows over 8 x 8192 keys: 81 us with 256, 50 with 512, 60 with 768, 54 with 1024),
// and no more (6 prompt chunks, 372 blocks of some 35 steps: 84 us whole, 88 in two).
constexpr int64_t kAttnSplitBlocks = 4096;
constexpr int64_t kAttnTileBlocks = 512;
// Fewest steps of a split: one for each wave of a split block (777 keys of one
// sequence: 10.4 us, 12.5 with half as many splits, 14.9 with a third), four of
// the tile kernel's, whose prologue takes as long (32 rows over 512 keys: 15.8 us,
// 18.8 with eight).
constexpr int64_t kAttnMinChunk = 4;
constexpr int64_t kAttnMostBlocks = (int64_t(1) << 24) - 1;
// Keys of the last steps, and of those that are looked up ahead, stay below 2^31.
constexpr int64_t kAttnMostKeys = INT32_MAX - 1024;
constexpr int64_t kAttnMaxWorkspace = int64_t(1) << 30;

int plan_attention(const kvstore_attention_args& a, const kvstore_paged_cache& c,
                   AttentionPlan* plan) {
  if (c.format < KVSTORE_FMT_BF16 || c.format > KVSTORE_FMT_FP4) return KVSTORE_ERR_DTYPE;
  if (a.src_dtype != KVSTORE_SRC_BF16 && a.src_dtype != KVSTORE_SRC_FP16) return KVSTORE_ERR_DTYPE;
  if (c.num_heads <= 0 || c.head_dim <= 0 || c.head_dim > 256 || a.q_heads <= 0 ||
      a.q_heads % c.num_heads || c.page_size <= 0 || c.page_size > INT32_MAX || c.num_slots <= 0 ||
      c.num_slots < c.page_size || c.num_slots / c.page_size > INT32_MAX || a.max_pages == 0 ||
      (int64_t)a.max_pages > kAttnMostKeys / c.page_size || a.max_len < 0 || a.window < 0 ||
      a.sinks < 0 || !(a.sm_scale >= 0.0f) || !(a.sm_scale <= 2.3e38f))
    return KVSTORE_ERR_SHAPE;
  if (a.cu_q == nullptr && a.tokens != a.seqs) return KVSTORE_ERR_SHAPE;
  if ((int64_t)a.tokens * a.q_heads > INT32_MAX) return KVSTORE_ERR_SHAPE;
  const int64_t group = a.q_heads / c.num_heads;
  const int64_t max_q = a.cu_q == nullptr ? 1 : a.max_q == 0 || a.max_q > a.tokens ? a.tokens : a.max_q;
  const int64_t rows = max_q * group;
  plan->max_keys = (int32_t)(a.max_pages * c.page_size);
  int64_t keys = a.max_len > 0 && a.max_len < plan->max_keys ? a.max_len : plan->max_keys;
  const int64_t seen = a.window > 0 && a.window < keys && a.sinks < keys - a.window ? a.window + a.sinks : keys;
  const bool sixteen = c.format == KVSTORE_FMT_BF16 || c.format == KVSTORE_FMT_FP16;
  plan->split = rows <= kvattn::kSplitRows &&
                !(sixteen && c.head_dim > 64 &&
                  seen > kAttnTileBytes / (4 * (int64_t)c.head_dim * c.num_heads) / a.seqs);
  const int64_t step = plan->split ? kvattn::kSplitStep : kvattn::kTileStep;
  plan->padded_dim = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
  const int64_t tile = plan->split ? kvattn::kSplitRows : kvattn::kTileRows;
  const int64_t slots = a.cu_q == nullptr ? a.seqs * ceil_div(group, tile)
                                          : (int64_t)a.tokens * group / tile + a.seqs;
  // blocks of 256 threads: a launch stays below 2^32 work-items (with its splits:
  // below)
  if ((slots + 7) * c.num_heads > kAttnMostBlocks) return KVSTORE_ERR_SHAPE;
  plan->tile_slots = (uint32_t)slots;
  // Steps of a tile, at most (a longer sequence than max_len gets longer splits).
  if (a.window > 0) {
    const int64_t span = a.window + (max_q < ceil_div(tile, group) ? max_q : ceil_div(tile, group)) +
                         a.sinks + 2 * step;
    if (a.window < keys && a.sinks < keys && span < keys) keys = span;
  }
  const int64_t steps = ceil_div(keys, step);
  const int64_t tiles = a.cu_q == nullptr ? slots
                        : rows <= tile    ? (int64_t)a.seqs
                                          : (int64_t)a.tokens * group / tile + a.seqs / 2;
  const int64_t whole = (tiles > 0 ? tiles : 1) * c.num_heads;   // blocks without splits
  int64_t splits = plan->split ? ceil_div(kAttnSplitBlocks, whole) : kAttnTileBlocks / whole;
  if (splits < 1) splits = 1;
  if (splits > ceil_div(steps, kAttnMinChunk)) splits = ceil_div(steps, kAttnMinChunk);
  const int64_t row_bytes = (int64_t)a.tokens * a.q_heads * (c.head_dim + 2) * 4;
  if (row_bytes > 0 && splits > kAttnMaxWorkspace / row_bytes) splits = kAttnMaxWorkspace / row_bytes;
  const int64_t room = (kAttnMostBlocks / c.num_heads - 7) / (slots > 0 ? slots : 1);
  if (splits > room) splits = room;
  // the kernel that joins splits has a block for every four rows of a tile
  plan->join_parts = (uint32_t)ceil_div(rows < tile ? rows : tile, 4);
  if (slots * c.num_heads > kAttnMostBlocks / plan->join_parts) splits = 1;
  if (splits > 256) splits = 256;
  if (splits < 1) splits = 1;
  plan->chunk_steps = (int32_t)(ceil_div(ceil_div(steps, splits), 4) * 4);
  splits = ceil_div(steps, plan->chunk_steps);
  plan->splits = (int32_t)(splits < 1 ? 1 : splits);
  // the sums, then (maximum, sum) pairs; both 16-byte aligned
  plan->workspace = plan->splits > 1 ? ceil_div(row_bytes * plan->splits, 16) * 16 : 0;
  return KVSTORE_OK;
}

kvattn::Side attention_side(const kvstore_paged_cache& c, bool is_v) {
  const CacheSide s = cache_side(c, is_v);
  return {s.data, s.page, s.offset, s.head, s.scales, s.s_page, s.s_offset, s.s_head};
}

}  // namespace

extern "C" {

int64_t kvstore_attention_workspace(const kvstore_attention_args* args,
                                    const kvstore_paged_cache* cache) {
  if (!args || !cache) return KVSTORE_ERR_NULL;
  if (args->tokens == 0 || args->seqs == 0) return 0;
  AttentionPlan plan;
  const int st = plan_attention(*args, *cache, &plan);
  return st != KVSTORE_OK ? st : plan.workspace;
}

int kvstore_attention_paged(const kvstore_attention_args* args, const kvstore_paged_cache* cache,
                            hipStream_t stream) {
  if (!args || !cache) return KVSTORE_ERR_NULL;
  const kvstore_attention_args& a = *args;
  const kvstore_paged_cache& c = *cache;
  if (a.src_dtype != KVSTORE_SRC_BF16 && a.src_dtype != KVSTORE_SRC_FP16) return KVSTORE_ERR_DTYPE;
  if (a.tokens == 0 || a.seqs == 0) return KVSTORE_OK;
  int st = check_paged_cache(c, true);
  if (st != KVSTORE_OK) return st;
  const bool fp16 = a.src_dtype == KVSTORE_SRC_FP16;
  const int fmt = row_fmt(c.format);
  if (fmt == kRow16 && fp16_format(c.format) != fp16) return KVSTORE_ERR_DTYPE;
  if (!a.q || !a.out || !a.page_table || !a.seq_lens) return KVSTORE_ERR_NULL;
  if (a.q == a.out) return KVSTORE_ERR_SHAPE;
  AttentionPlan plan;
  st = plan_attention(a, c, &plan);
  if (st != KVSTORE_OK) return st;
  st = check_row_strides(a.q_stride_token, a.q_stride_head, a.q_heads, c.head_dim, a.tokens);
  if (st != KVSTORE_OK) return st;
  st = check_row_strides(a.o_stride_token, a.o_stride_head, a.q_heads, c.head_dim, a.tokens);
  if (st != KVSTORE_OK) return st;
  if (a.table_stride < 0 || !fits((int64_t)a.seqs + 1, a.table_stride) ||
      !sum_fits((int64_t)a.seqs * a.table_stride, a.max_pages, 0))
    return KVSTORE_ERR_SHAPE;
  if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.page_table, 4) ||
      !aligned(a.seq_lens, 4) || !aligned(a.cu_q, 4))
    return KVSTORE_ERR_ALIGN;
  if (plan.workspace > 0) {
    if (!a.workspace) return KVSTORE_ERR_NULL;
    if (!aligned(a.workspace, 16)) return KVSTORE_ERR_ALIGN;
    if (a.workspace_bytes < plan.workspace) return KVSTORE_ERR_SHAPE;
  }
  kvattn::Params p;
  p.flag = error_flag();
  if (!p.flag) return KVSTORE_ERR_HIP;
  p.q = static_cast<const uint8_t*>(a.q);
  p.out = static_cast<uint8_t*>(a.out);
  p.q_token = a.q_stride_token;
  p.q_head = a.q_stride_head;
  p.o_token = a.o_stride_token;
  p.o_head = a.o_stride_head;
  p.cu_q = a.cu_q;
  p.table = a.page_table;
  p.seq_lens = a.seq_lens;
  p.table_stride = a.table_stride;
  p.k = attention_side(c, false);
  p.v = attention_side(c, true);
  p.ws_o = static_cast<float*>(a.workspace);
  p.ws_ml = p.ws_o ? p.ws_o + (int64_t)a.tokens * a.q_heads * plan.splits * c.head_dim : nullptr;
  p.tokens = a.tokens;
  p.seqs = a.seqs;
  p.tile_slots = plan.tile_slots;
  p.kv_heads = (uint32_t)c.num_heads;
  p.group = (uint32_t)(a.q_heads / c.num_heads);
  p.dim = c.head_dim;
  p.page_size = (int32_t)c.page_size;
  p.page_shift = page_shift_of(c.page_size);
  p.num_pages = (int32_t)(c.num_slots / c.page_size);
  p.max_keys = plan.max_keys;
  p.window = a.window == 0 || a.window > INT32_MAX ? INT32_MAX : (int32_t)a.window;
  p.sinks = a.sinks > INT32_MAX ? INT32_MAX : (int32_t)a.sinks;
  p.scale2 = a.sm_scale * 1.44269504088896340736f;
  p.scale_kind = c.scale_kind;
  p.chunk_steps = plan.chunk_steps;
  p.splits = plan.splits;
  p.join_parts = plan.join_parts;
  static const kvattn::Launch split[2][4] = {
      {kvattn::launch_split_bf16_0, kvattn::launch_split_bf16_1, kvattn::launch_split_bf16_2,
       kvattn::launch_split_bf16_3},
      {kvattn::launch_split_fp16_0, kvattn::launch_split_fp16_1, kvattn::launch_split_fp16_2,
       kvattn::launch_split_fp16_3}};
  static const kvattn::Launch tile[2][4] = {
      {kvattn::launch_tile_bf16_0, kvattn::launch_tile_bf16_1, kvattn::launch_tile_bf16_2,
       kvattn::launch_tile_bf16_3},
      {kvattn::launch_tile_fp16_0, kvattn::launch_tile_fp16_1, kvattn::launch_tile_fp16_2,
       kvattn::launch_tile_fp16_3}};
  return (plan.split ? split : tile)[fp16][fmt](p, plan.padded_dim, stream);
}

}  // extern "C"
