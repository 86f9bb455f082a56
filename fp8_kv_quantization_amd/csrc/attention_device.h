// Device code that the attention kernels share: which rows and keys a block
// works on, and the conversions of cached values to 16 bits.
#pragma once

#include "attention.h"

namespace kvattn {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ void report(unsigned long long* flag, uint32_t token) {
  unsigned long long seen = 0xFFFFFFFFull;
  for (;;) {   // ends: every failed exchange means that another report landed
    const uint32_t first = (uint32_t)seen < token ? (uint32_t)seen : token;
    const uint32_t count = (uint32_t)(seen >> 32);
    const unsigned long long next =
        ((unsigned long long)(count == 0xFFFFFFFFu ? count : count + 1u) << 32) | first;
    const unsigned long long prev = atomicCAS(flag, seen, next);
    if (prev == seen) return;
    seen = prev;
  }
}

__device__ __forceinline__ int32_t clamp_row(const Params& p, int32_t r) {
  return r < 0 ? 0 : (uint32_t)r > p.tokens ? (int32_t)p.tokens : r;
}

// Tile slots: sequence b of new-token rows [c_b, c_{b+1}) owns the slots from
// c_b * group / rows + b on.  These starts grow by at least one per sequence
// and leave it room for all its tiles (floor(x + y) >= floor(x) + ceil(y) - 1),
// so a block finds its sequence from cu_q alone, with no prefix sums; slots
// beyond a sequence's tiles hold nothing.
// A tile: `rows` (token, head in group) pairs of one sequence, and its keys as
// steps of kStep: first those of the first tokens, then those of the window.
template <int kStep>
struct Tile {
  uint32_t seq;
  int32_t token0;      // row of q of the tile's first token
  int32_t row0, rows;  // rows [row0, row0 + rows) of the sequence's new tokens * group
  int32_t first_pos;   // position of the sequence's first new token
  int32_t p_lo, p_hi;  // positions of the tile's first and last token
  int32_t end;         // keys are [0, end)
  int32_t low;         // first key of any row's window
  int32_t sink_steps;  // steps [0, sink_steps) start at key 0
  int32_t low_step;    // step sink_steps starts at key low_step * kStep
  int32_t steps;

  __device__ __forceinline__ int32_t key_of(int32_t step) const {
    return (step < sink_steps ? step : step - sink_steps + low_step) * kStep;
  }
};

// Steps of a split of the tile, and how many splits that makes (at least one).
// A tile with more steps than the host planned for gets longer splits.
template <int kStep>
__device__ __forceinline__ int32_t split_steps(const Params& p, const Tile<kStep>& t,
                                               int32_t* n_splits) {
  const int32_t even = (t.steps + p.splits - 1) / p.splits;
  const int32_t chunk = even > p.chunk_steps ? even : p.chunk_steps;
  *n_splits = t.steps <= chunk ? 1 : (t.steps + chunk - 1) / chunk;
  return chunk;
}

__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// False where the slot holds no tile.  All lanes of a wave call it together.
template <int kStep>
__device__ __forceinline__ bool tile_of(const Params& p, uint32_t slot, int32_t tile_rows,
                                        Tile<kStep>* t) {
  int32_t begin, n, len;
  int32_t index;   // of the tile in its sequence
  if (p.cu_q == nullptr) {
    const uint32_t per = (p.group + tile_rows - 1) / tile_rows;
    t->seq = slot / per;
    index = slot - t->seq * per;
    begin = t->seq;
    n = 1;
    len = uniform(p.seq_lens[t->seq]);
  } else {
    // The last sequence whose start is at most `slot`, by 64-way search: starts
    // increase, so the lanes that hold one at most `slot` are the first ones.
    // The last round, over neighbours, has what the tile needs in its lanes.
    const uint32_t lane = threadIdx.x & 63;
    uint32_t lo = 0, size = p.seqs;
    for (;;) {
      const uint32_t stride = (size + 63) / 64;
      const uint32_t at = lane * stride, b = lo + (at < size ? at : size - 1);
      const int32_t c0 = clamp_row(p, p.cu_q[b]), c1 = clamp_row(p, p.cu_q[b + 1]);
      const int32_t keys = p.seq_lens[b];
      const int64_t start = (int64_t)c0 * p.group / tile_rows + b;
      const uint32_t k = __popcll(__ballot(at < size && start <= slot));
      if (k == 0) return false;   // before the first sequence
      if (stride == 1) {
        t->seq = uniform(lo + k - 1);
        begin = __builtin_amdgcn_readlane(c0, k - 1);
        n = __builtin_amdgcn_readlane(c1, k - 1) - begin;
        len = __builtin_amdgcn_readlane(keys, k - 1);
        const int64_t i = (int64_t)slot - ((int64_t)begin * p.group / tile_rows + t->seq);
        if (n <= 0 || i * tile_rows >= (int64_t)n * p.group) return false;
        index = (int32_t)i;
        break;
      }
      lo = uniform(lo + (k - 1) * stride);
      const uint32_t rest = size - (k - 1) * stride;
      size = uniform(rest < stride ? rest : stride);
    }
  }
  len = len < 0 ? 0 : len > p.max_keys ? p.max_keys : len;
  const int64_t all = (int64_t)n * p.group;
  const int64_t r0 = (int64_t)index * tile_rows;
  // rows of a sequence stay below 2^31: checked on the host (tokens * group)
  t->row0 = (int32_t)r0;
  t->rows = (int32_t)(all - r0 < tile_rows ? all - r0 : tile_rows);
  t->token0 = begin;
  t->first_pos = len - n;
  t->p_lo = t->first_pos + t->row0 / (int32_t)p.group;
  t->p_hi = t->first_pos + (t->row0 + t->rows - 1) / (int32_t)p.group;
  t->end = t->p_hi + 1;   // p_hi < len
  if (t->end <= 0) {      // positions before the sequence: no keys
    t->end = t->low = t->sink_steps = t->low_step = t->steps = 0;
    return true;
  }
  const int64_t low = (int64_t)t->p_lo - p.window + 1;
  t->low = low > 0 ? (int32_t)low : 0;
  t->low_step = t->low / kStep;
  const int32_t sinks = p.sinks < t->low_step * kStep ? p.sinks : t->low_step * kStep;
  t->sink_steps = (sinks + kStep - 1) / kStep;
  t->steps = t->sink_steps + (t->end + kStep - 1) / kStep - t->low_step;
  return true;
}

// Conversions of cached codes to pairs of the source type; values are exact
// (code * 2^e) as far as the type's range goes.
template <bool kFp16, int kFmt>
__device__ __forceinline__ uint32_t pair_of8(uint32_t w, float scale, bool hi) {
  if constexpr (kFp16) {
    h16x2 r;
    if constexpr (kFmt == kFmtE4M3)
      r = hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true)
             : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false);
    else
      r = hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, scale, true)
             : __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, scale, false);
    return __builtin_bit_cast(uint32_t, r);
  } else {
    b16x2 r;
    if constexpr (kFmt == kFmtE4M3)
      r = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true)
             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
    else
      r = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, true)
             : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, false);
    return __builtin_bit_cast(uint32_t, r);
  }
}

template <bool kFp16, int kSel>
__device__ __forceinline__ uint32_t pair_of4(uint32_t w, float scale) {
  if constexpr (kFp16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, kSel));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, kSel));
}

// Eight cached elements -> eight 16-bit values.  `w`: 16 bytes (16 bits), the
// first 8 (FP8) or 4 (4 bits) of them.
template <bool kFp16, int kFmt>
__device__ __forceinline__ u32x4 values8(uint32_t w0, uint32_t w1, float scale) {
  if constexpr (kFmt == kFmtFp4)
    return u32x4{pair_of4<kFp16, 0>(w0, scale), pair_of4<kFp16, 1>(w0, scale),
                 pair_of4<kFp16, 2>(w0, scale), pair_of4<kFp16, 3>(w0, scale)};
  else
    return u32x4{pair_of8<kFp16, kFmt>(w0, scale, false), pair_of8<kFp16, kFmt>(w0, scale, true),
                 pair_of8<kFp16, kFmt>(w1, scale, false), pair_of8<kFp16, kFmt>(w1, scale, true)};
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (kFp16) return __builtin_bit_cast(uint32_t, h16x2{(_Float16)a, (_Float16)b});
  else return __builtin_bit_cast(uint32_t, b16x2{(__bf16)a, (__bf16)b});
}

template <bool kFp16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (kFp16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h16x8, a),
                                                  __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, a),
                                                   __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
}

template <bool kFp16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (kFp16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, a),
                                                  __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, a),
                                                   __builtin_bit_cast(b16x8, b), c, 0, 0, 0);
}

// Four rows' 16-bit values of one column: lane i of a group of 16 addresses row
// i / 4, columns 4 * (i % 4) ... + 3 of a 4 x 16 block in LDS, and gets column
// i of its four rows.
__device__ __forceinline__ u32x2 read_column4(uint8_t* at) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
}

// Loads from addresses that went through LDS: as global memory, not generic.
template <typename T>
__device__ __forceinline__ T load_global(uint64_t at) {
  return *reinterpret_cast<__attribute__((address_space(1))) const T*>(at);
}

// 16 bytes a lane from global memory to LDS, at the wave's place plus 16 times
// the lane (counted by vmcnt).
__device__ __forceinline__ void load_to_lds(uint64_t from, uint8_t* wave_place) {
  __builtin_amdgcn_global_load_lds(
      reinterpret_cast<__attribute__((address_space(1))) void*>(from),
      (__attribute__((address_space(3))) void*)wave_place, 16, 0, 0);
}

// Non-finite 16-bit values of a pair replaced by zeros, or kept alone.
template <bool kFp16>
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, bool* special) {
  constexpr uint32_t e = kFp16 ? 0x7C00u : 0x7F80u;
  const bool lo = (w & e) == e, hi = (w & (e << 16)) == e << 16;
  *special = *special || lo || hi;
  return w & ~((lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u));
}
template <bool kFp16>
__device__ __forceinline__ u32x4 finite8(u32x4 w, bool* special) {
  return u32x4{finite_pair<kFp16>(w.x, special), finite_pair<kFp16>(w.y, special),
               finite_pair<kFp16>(w.z, special), finite_pair<kFp16>(w.w, special)};
}

// Element d of a cached V row, as a float; finite values give 0.  For the rare
// rows that see a NaN or an infinity (see the kernels' "special" passes).
template <int kFmt, bool kFp16>
__device__ __forceinline__ float special_at(const Params& p, uint32_t head, int32_t page,
                                            int32_t off, int32_t d) {
  const uint8_t* row = p.v.data + (int64_t)page * p.v.page + (int64_t)off * p.v.offset +
                       (int64_t)head * p.v.head;
  const uint8_t* sc = p.v.scales + (int64_t)page * p.v.s_page + (int64_t)off * p.v.s_offset;
  float x;
  if constexpr (kFmt == kFmt16) {
    const uint16_t w = reinterpret_cast<const uint16_t*>(row)[d];
    x = kFp16 ? (float)__builtin_bit_cast(_Float16, w) : __uint_as_float((uint32_t)w << 16);
  } else if constexpr (kFmt == kFmtFp4) {
    x = sc[(int64_t)head * p.v.s_head + d / 32] == 255 ? __builtin_nanf("") : 0.0f;
  } else {
    const uint32_t w = row[d];
    const float y = kFmt == kFmtE4M3 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 0)
                                     : __builtin_amdgcn_cvt_f32_bf8((int)w, 0);
    x = p.scale_kind == KVATTN_TENSOR
            ? y
            : y * *reinterpret_cast<const float*>(
                      sc + (p.scale_kind == KVATTN_TOKEN_HEAD ? (int64_t)head * p.v.s_head : 0));
  }
  return __builtin_isfinite(x) ? 0.0f : x;
}

// Page and offset of a key.
__device__ __forceinline__ void key_page(const Params& p, int32_t key, int32_t* page,
                                         int32_t* off) {
  if (p.page_shift >= 0) {
    *page = key >> p.page_shift;
    *off = key & (p.page_size - 1);
  } else {
    *page = (int32_t)((uint32_t)key / (uint32_t)p.page_size);
    *off = key - *page * p.page_size;
  }
}

// What a row of new tokens sees.
__device__ __forceinline__ bool sees(const Params& p, int32_t pos, int32_t key) {
  return key <= pos && (pos - key < p.window || key < p.sinks);
}

// Bits 0 ... n - 1 (none below 1, all from 64 on).
__device__ __forceinline__ unsigned long long low_bits(int32_t n) {
  const unsigned long long some = (1ull << (n & 63)) - 1ull;
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : some;
}

// sees() for the keys key0 + j of a step, as bits j: those that are there, at
// most pos, and inside the window or among the first tokens.
__device__ __forceinline__ unsigned long long seen_bits(const Params& p, int32_t pos, int32_t key0,
                                                        unsigned long long ok) {
  const int32_t last = pos - key0;   // >= -2^31 + 1: positions are above -2^31 / 2
  const unsigned long long behind = last < p.window ? 0ull : low_bits(last - p.window + 1);
  return ok & low_bits(last < 64 ? last + 1 : 64) &
         (~behind | low_bits(p.sinks < key0 ? 0 : p.sinks - key0));
}

// A row of a tile: its token (row of q), q head, and index among all rows.
struct Row {
  int64_t token;
  int32_t head;
  int64_t index;
};
template <int kStep>
__device__ __forceinline__ Row row_of(const Params& p, const Tile<kStep>& t, uint32_t kv_head,
                                      int32_t r) {
  const int32_t row = t.row0 + r, tok = row / (int32_t)p.group;
  Row x;
  x.token = t.token0 + tok;
  x.head = kv_head * p.group + (row - tok * (int32_t)p.group);
  x.index = x.token * (int64_t)(p.kv_heads * p.group) + x.head;
  return x;
}

// Joins the splits of a row, by a wave, in one pass: its loads wait for nothing
// but the sequence's length.
template <bool kFp16>
__device__ __forceinline__ void join_row(const Params& p, const Row& x, int32_t n_splits,
                                         float v_scale) {
  const int64_t at = x.index * p.splits;
  const int32_t lane = threadIdx.x & 63;
  // lanes: four dims of a split each, as many splits side by side as fit
  const int32_t quads = p.dim / 4, side = 64 / quads;
  const int32_t d = lane % quads * 4, first = lane / quads;
  float top = kNegInf, sum = 0.0f;
  f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kAtOnce = 4;
  if (first < side) {
    for (int32_t i0 = first; i0 < n_splits; i0 += kAtOnce * side) {
      float mi[kAtOnce], li[kAtOnce];
      f32x4 o[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int32_t i = i0 + e * side;
        const int64_t from = at + (i < n_splits ? i : i0);
        const f32x2 ml = *reinterpret_cast<const f32x2*>(p.ws_ml + 2 * from);
        mi[e] = i < n_splits ? ml.x : kNegInf;
        li[e] = ml.y;
        o[e] = *reinterpret_cast<const f32x4*>(p.ws_o + from * p.dim + d);
      }
      float now = top;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) now = fmaxf(now, mi[e]);
      const float keep = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - now);
      top = now;
      sum *= keep;
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] *= keep;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const float f = mi[e] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mi[e] - now);
        sum += mi[e] == kNegInf ? 0.0f : li[e] * f;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] += mi[e] == kNegInf ? 0.0f : o[e][j] * f;
      }
    }
  }
  if (side > 1) {   // the other splits' lanes, in order
    float all = top;
    for (int32_t k = 0; k < side; ++k) all = fmaxf(all, __shfl(top, lane % quads + k * quads));
    const float f = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - all);
    const float own_sum = sum * f;
    const f32x4 own = f32x4{y[0] * f, y[1] * f, y[2] * f, y[3] * f};
    sum = 0.0f;
    y = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int32_t k = 0; k < side; ++k) {
      const int32_t from = lane % quads + k * quads;
      sum += __shfl(own_sum, from);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] += __shfl(own[j], from);
    }
  }
  if (first > 0) return;
  const float inv = sum == 0.0f ? 0.0f : v_scale / sum;
  *reinterpret_cast<u32x2*>(p.out + x.token * p.o_token + (int64_t)x.head * p.o_head + 2 * d) =
      u32x2{pack_pair<kFp16>(y[0] * inv, y[1] * inv), pack_pair<kFp16>(y[2] * inv, y[3] * inv)};
}

// Joins the splits of each row, kJoinRows rows a block at a time.
constexpr int kJoinRows = 4;
template <bool kFp16, int kStep>
__device__ __forceinline__ void join_splits(const Params& p, int32_t tile_rows, float v_scale) {
  const uint32_t part = blockIdx.x % p.join_parts, turn = blockIdx.x / p.join_parts;
  const uint32_t head = turn % p.kv_heads, slot = turn / p.kv_heads;
  Tile<kStep> t;
  if (!tile_of(p, slot, tile_rows, &t)) return;
  int32_t n_splits;
  split_steps(p, t, &n_splits);
  if (n_splits == 1) return;
  // more rows than the host was told of take further turns
  for (int32_t r = part * kJoinRows + uniform(threadIdx.x >> 6); r < t.rows;
       r += p.join_parts * kJoinRows)
    join_row<kFp16>(p, row_of(p, t, head, r), n_splits, v_scale);
}

}  // namespace kvattn
