// Rotated append into a paged cache and load out of it (include/kvstore_paged.h).
// Part of the translation unit of libkvstore.hip, after kvstore.hip, whose
// error flag, conversions, checks and launch helper it uses.
//
// Both operators are data movement, bound by HBM: a token's heads are read
// once, converted in registers and written once.  A lane works on one 8-element
// chunk (16 bytes of 16-bit values) of kHeads consecutive heads of a token, so
// a wave access covers whole 128-byte lines of each head.
//
// Measured: 16384 tokens of 32 q and 8 kv heads of 128 bf16 dims, rotated, into an
// e4m3fn cache (378 MB) 69 us, 5.5 TB/s (a large device copy reaches 4.9); 8192
// into a 4-bit cache and back out 49.7 us for 224 MB (42 and 10 us); 16384 rows of 8
// heads out of an e4m3fn cache with a scale for each token and head (102 MB) 21
// us; 16 tokens of a decode step 3.4 us, the cost of a launch.

#include "kvstore_paged.h"

namespace {

constexpr int kRowsWaves = 4;   // waves per block

// Element formats as the kernels see them: 16-bit (of the source type), e4m3fn,
// e5m2, 4-bit blocks.
enum RowFmt { kRow16 = 0, kRowE4M3 = 1, kRowE5M2 = 2, kRowFp4 = 3 };

struct CacheSide {   // K or V of a paged cache
  uint8_t* data;
  int64_t page, offset, head;
  uint8_t* scales;
  int64_t s_page, s_offset, s_head;
};

struct RowsParams {
  CacheSide k_side, v_side;
  const void* indices;
  int64_t idx_stride;
  int64_t num_slots, page_size;
  int32_t page_shift;       // log2(page_size) when a power of two, else -1
  int32_t idx64;
  uint32_t batch, token_base;
  uint32_t chunks;          // head_dim / 8
  uint32_t heads_per_wave;  // 64 / chunks: heads whose chunks a wave access covers
  uint32_t groups;          // groups of kHeads heads per token
};

// Slot -> page and offset, by shift, or by 32-bit division where the numbers fit.
__device__ __forceinline__ void page_of(int64_t loc, int64_t page_size, int32_t page_shift,
                                        int64_t* page, int64_t* off) {
  if (page_shift >= 0) {
    *page = loc >> page_shift;
    *off = loc & (page_size - 1);
  } else if (((uint64_t)loc | (uint64_t)page_size) >> 32 == 0) {
    const uint32_t q = (uint32_t)loc / (uint32_t)page_size;
    *page = q;
    *off = (uint32_t)loc - q * (uint32_t)page_size;
  } else {
    *page = loc / page_size;
    *off = loc - *page * page_size;
  }
}

__device__ __forceinline__ int64_t index_at(const void* p, int64_t at, int is64) {
  return is64 ? static_cast<const int64_t*>(p)[at] : (int64_t)static_cast<const int32_t*>(p)[at];
}

// What a lane of a rows kernel works on: the chunk c of the heads
// [group * kHeads, ...) of a token.  Lanes past the last whole head of the wave,
// or past the batch, repeat the last unit and store nothing, so every lane
// takes part in the cross-lane steps.
struct RowsLane {
  uint32_t token;   // of the whole batch
  uint32_t group, c;
  bool active;
};

__device__ __forceinline__ RowsLane rows_lane(const RowsParams& p) {
  const uint32_t lane = threadIdx.x % kWave;
  const uint32_t wave = blockIdx.x * kRowsWaves + threadIdx.x / kWave;
  const uint32_t hl = lane / p.chunks;
  const uint32_t units = p.batch * p.groups;   // < 2^31 by the launch's token runs
  const uint32_t unit = wave * p.heads_per_wave + hl;
  RowsLane r;
  r.active = hl < p.heads_per_wave && unit < units;
  const uint32_t u = unit < units ? unit : units - 1;
  const uint32_t t = u / p.groups;
  r.c = lane - hl * p.chunks;
  r.group = u - t * p.groups;
  r.token = p.token_base + t;
  return r;
}

template <bool kFp16>
__device__ __forceinline__ void widen8(u32x4 a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = kFp16 ? f16_lo(w[i]) : bf16_lo(w[i]);
    x[2 * i + 1] = kFp16 ? f16_hi(w[i]) : bf16_hi(w[i]);
  }
}

// Two fp32 values rounded to nearest even, the first in the low half.
template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kFp16) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
  } else {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, b2{(__bf16)a, (__bf16)b});
  }
}

template <bool kFp16>
__device__ __forceinline__ u32x4 pack8(const float (&y)[8]) {
  return u32x4{pack2<kFp16>(y[0], y[1]), pack2<kFp16>(y[2], y[3]), pack2<kFp16>(y[4], y[5]),
               pack2<kFp16>(y[6], y[7])};
}

// Eight scaled fp32 values -> FP8 codes: converted unclamped, and again on the
// exact path where that leaves a NaN or infinity code (see quantize16_checked).
template <bool kE5M2>
__device__ __forceinline__ u32x2 fp8_of8(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
  u32x2 q;
  q.x = (uint32_t)cvt_pk<kE5M2>(y[2], y[3], cvt_pk<kE5M2>(y[0], y[1], 0, false), true);
  q.y = (uint32_t)cvt_pk<kE5M2>(y[6], y[7], cvt_pk<kE5M2>(y[4], y[5], 0, false), true);
  const bool special = any_special<kE5M2>(u32x4{q.x, q.y, 0u, 0u});
  if (__builtin_expect(__ballot(special) != 0, 0)) {
    if (special) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = scale_sat<kE5M2>(x[i], inv);
      q.x = pack_fp8<kE5M2>(y[0], y[1], y[2], y[3]);
      q.y = pack_fp8<kE5M2>(y[4], y[5], y[6], y[7]);
    }
  }
  return q;
}

// Scale byte of a 32-element block from the largest magnitude's bit pattern
// (patterns of magnitudes order like the magnitudes, NaN above infinity): the
// smallest power of two with amax <= 7 scales is 2^(e - 2), or 2^(e - 1) where
// the significand exceeds 1.75.
constexpr uint32_t kFp4MinScale = 27;   // 2^-100: every value code * scale is a normal number
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  const uint32_t e = (amax >> 23) + ((amax & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  return e < kFp4MinScale + 2 ? kFp4MinScale : e - 2;
}

// Eight values -> eight e2m1 codes (round to nearest even, saturating to 6).
__device__ __forceinline__ uint32_t fp4_of8(const float (&y)[8], uint32_t byte) {
  if (byte == 255u) return 0u;
  const float scale = __uint_as_float(byte << 23);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[0], y[1], scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[2], y[3], scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[4], y[5], scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[6], y[7], scale, 3);
  return q;
}

// ---------------------------------------------------------------------------
// Rotated append.
// ---------------------------------------------------------------------------
struct RopeParams {
  RowsParams rows;
  const uint8_t *q, *k, *v;
  uint8_t* q_out;
  int64_t q_token, q_head, qo_token, qo_head, k_token, k_head, v_token, v_head;
  const void* positions;
  const uint8_t* cos_sin;
  int64_t cos_sin_stride, num_positions;
  const float *inv_k, *inv_v;
  uint32_t q_heads, kv_heads;
  uint32_t rot;       // rotated dims
  int32_t pos64;
};

// A product rounded on its own.  The compiler would fuse it into the sum that
// takes it (v_fma_mix_f32), which gives other last bits, and so now and then
// another code, than the operator's definition.
__device__ __forceinline__ float product(float a, float b) {
  float x = a * b;
  asm volatile("" : "+v"(x));
  return x;
}

enum RopeKind { kNoRope = 0, kHalves = 1, kInterleaved = 2 };

// Heads of a token are numbered q, then k, then v.  A lane's partner chunk
// (the other half's dims) is loaded too: it comes out of the cache line's
// other reader in the same wave, and it lets every lane write its own chunk
// whatever rot_dim is.  Loads of all heads come before the first store, and a
// wave holds whole heads, so q_out may be q.
template <bool kFp16, int kFmt, int kRope, int kHeads>
__global__ __launch_bounds__(kWave * kRowsWaves) void kvstore_rope_kernel(const RopeParams p) {
  const RowsParams& r = p.rows;
  const RowsLane L = rows_lane(r);
  const int64_t token = L.token;
  const int64_t loc = index_at(r.indices, token * r.idx_stride, r.idx64);
  const uint32_t d = 8 * L.c, half = p.rot / 2;
  const bool turned = kRope != kNoRope && d < p.rot;
  bool pos_ok = true;
  float cs[8], sn[8];
  if constexpr (kRope != kNoRope) {
    int64_t pos = index_at(p.positions, token, p.pos64);
    pos_ok = pos >= 0 && pos < p.num_positions;
    const float* row =
        reinterpret_cast<const float*>(p.cos_sin + (pos_ok ? pos : 0) * p.cos_sin_stride);
    constexpr int n = kRope == kInterleaved ? 4 : 8;
    const uint32_t at = !turned ? 0 : kRope == kInterleaved ? d / 2 : d < half ? d : d - half;
#pragma unroll
    for (int i = 0; i < n; i += 4) {
      *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(row + at + i);
      *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(row + half + at + i);
    }
  }
  // byte distance to the partner chunk
  const int32_t apart = kRope == kHalves && turned ? (d < half ? 2 * (int)half : -2 * (int)half) : 0;

  const uint32_t total = p.q_heads + 2 * p.kv_heads;
  const uint32_t h0 = L.group * kHeads;
  u32x4 own[kHeads], other[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const uint32_t h = h0 + j < total ? h0 + j : total - 1;
    const uint8_t* src = h < p.q_heads ? p.q + token * p.q_token + (int64_t)h * p.q_head
                         : h < p.q_heads + p.kv_heads
                             ? p.k + token * p.k_token + (int64_t)(h - p.q_heads) * p.k_head
                             : p.v + token * p.v_token +
                                   (int64_t)(h - p.q_heads - p.kv_heads) * p.v_head;
    own[j] = *reinterpret_cast<const u32x4*>(src + 2 * d);
    if constexpr (kRope == kHalves) other[j] = *reinterpret_cast<const u32x4*>(src + 2 * d + apart);
  }

  const bool in_range = loc >= 0 && loc < r.num_slots;
  int64_t page, off;
  page_of(in_range ? loc : 0, r.page_size, r.page_shift, &page, &off);
  const float inv_k = kFmt == kRowE4M3 || kFmt == kRowE5M2 ? (p.inv_k ? *p.inv_k : 1.0f) : 1.0f;
  const float inv_v = kFmt == kRowE4M3 || kFmt == kRowE5M2 ? (p.inv_v ? *p.inv_v : 1.0f) : 1.0f;
  if (L.active && !(in_range && pos_ok) && h0 == 0 && L.c == 0) report_bad_token(L.token);

#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const uint32_t h = h0 + j;
    const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.kv_heads;
    float x[8];
    widen8<kFp16>(own[j], x);
    bool changed = false;
    if constexpr (kRope == kHalves) {
      if (turned && !is_v) {
        float o[8];
        widen8<kFp16>(other[j], o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = product(x[i], cs[i]), b = product(o[i], sn[i]);
          x[i] = d < half ? a - b : a + b;
        }
        changed = true;
      }
    }
    if constexpr (kRope == kInterleaved) {
      if (turned && !is_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = product(a, cs[i]) - product(b, sn[i]);
          x[2 * i + 1] = product(b, cs[i]) + product(a, sn[i]);
        }
        changed = true;
      }
    }
    const bool live = L.active && pos_ok && h < total;
    const u32x4 bits = changed ? pack8<kFp16>(x) : own[j];
    if (is_q) {
      if (live)
        *reinterpret_cast<u32x4*>(p.q_out + token * p.qo_token + (int64_t)h * p.qo_head + 2 * d) =
            bits;
    }
    const bool store = live && in_range && !is_q;
    const uint32_t hk = is_v ? h - p.q_heads - p.kv_heads : h - p.q_heads;
    const CacheSide& s = is_v ? r.v_side : r.k_side;
    uint8_t* slot = s.data + page * s.page + off * s.offset + (int64_t)hk * s.head;
    if constexpr (kFmt == kRow16) {
      if (store) *reinterpret_cast<u32x4*>(slot + 2 * d) = bits;
    } else if constexpr (kFmt == kRowFp4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
      m = dpp_max<0x4E>(dpp_max<0xB1>(m));   // the four lanes of the 32-element block
      const uint32_t byte = fp4_scale_byte(m);
      const uint32_t codes = fp4_of8(x, byte);
      if (store) {
        *reinterpret_cast<uint32_t*>(slot + d / 2) = codes;
        if ((L.c & 3) == 0)
          s.scales[page * s.s_page + off * s.s_offset + (int64_t)hk * s.s_head + L.c / 4] =
              (uint8_t)byte;
      }
    } else {
      const u32x2 codes = fp8_of8<kFmt == kRowE5M2>(x, is_v ? inv_v : inv_k);
      if (store) *reinterpret_cast<u32x2*>(slot + d) = codes;
    }
  }
}

// ---------------------------------------------------------------------------
// Load.
// ---------------------------------------------------------------------------
struct LoadParams {
  RowsParams rows;
  uint8_t *k_out, *v_out;
  int64_t ko_token, ko_head, vo_token, vo_head;
  const float *k_scale, *v_scale;   // KVSTORE_SCALES_TENSOR, nullable
  uint32_t kv_heads;
  int32_t scale_kind;
};

template <int kFmt>
__device__ __forceinline__ void fp8_values8(u32x2 q, float (&x)[8]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f2 lo = kFmt == kRowE5M2 ? __builtin_amdgcn_cvt_pk_f32_bf8((int)w[i], false)
                                   : __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
    const f2 hi = kFmt == kRowE5M2 ? __builtin_amdgcn_cvt_pk_f32_bf8((int)w[i], true)
                                   : __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    x[4 * i] = lo.x; x[4 * i + 1] = lo.y; x[4 * i + 2] = hi.x; x[4 * i + 3] = hi.y;
  }
}

__device__ __forceinline__ void fp4_values8(uint32_t q, float scale, float (&x)[8]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 0);
  const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 1);
  const f2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 2);
  const f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 3);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}

// Heads of a token are numbered k, then v.
template <bool kFp16, int kFmt, int kHeads>
__global__ __launch_bounds__(kWave * kRowsWaves) void kvstore_load_kernel(const LoadParams p) {
  const RowsParams& r = p.rows;
  const RowsLane L = rows_lane(r);
  const int64_t token = L.token;
  const int64_t loc = index_at(r.indices, token * r.idx_stride, r.idx64);
  const bool in_range = loc >= 0 && loc < r.num_slots;
  int64_t page, off;
  page_of(in_range ? loc : 0, r.page_size, r.page_shift, &page, &off);
  const uint32_t d = 8 * L.c, total = 2 * p.kv_heads, h0 = L.group * kHeads;

  u32x4 raw[kHeads];
  float scale[kHeads];
  uint32_t byte[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const uint32_t h = h0 + j < total ? h0 + j : total - 1;
    const bool is_v = h >= p.kv_heads;
    const int64_t hk = is_v ? h - p.kv_heads : h;
    const CacheSide& s = is_v ? r.v_side : r.k_side;
    const uint8_t* slot = s.data + page * s.page + off * s.offset + hk * s.head;
    const uint8_t* sc = s.scales + page * s.s_page + off * s.s_offset;
    if constexpr (kFmt == kRow16) {
      raw[j] = *reinterpret_cast<const u32x4*>(slot + 2 * d);
    } else if constexpr (kFmt == kRowFp4) {
      raw[j].x = *reinterpret_cast<const uint32_t*>(slot + d / 2);
      byte[j] = sc[hk * s.s_head + L.c / 4];
    } else {
      const u32x2 q = *reinterpret_cast<const u32x2*>(slot + d);
      raw[j].x = q.x;
      raw[j].y = q.y;
      if (p.scale_kind == KVSTORE_SCALES_TENSOR) {
        const float* one = is_v ? p.v_scale : p.k_scale;
        scale[j] = one ? *one : 1.0f;
      } else {
        scale[j] = *reinterpret_cast<const float*>(
            sc + (p.scale_kind == KVSTORE_SCALES_TOKEN_HEAD ? hk * s.s_head : 0));
      }
    }
  }
  if (L.active && !in_range && h0 == 0 && L.c == 0) report_bad_token(L.token);
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const uint32_t h = h0 + j;
    const bool is_v = h >= p.kv_heads;
    u32x4 out;
    float x[8];
    if constexpr (kFmt == kRow16) {
      out = raw[j];
    } else if constexpr (kFmt == kRowFp4) {
      fp4_values8(raw[j].x, __uint_as_float(byte[j] << 23), x);
      out = pack8<kFp16>(x);
    } else {
      fp8_values8<kFmt>(u32x2{raw[j].x, raw[j].y}, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], scale[j]);
      out = pack8<kFp16>(x);
    }
    if (L.active && in_range && h < total) {
      uint8_t* dst = is_v ? p.v_out + token * p.vo_token + (int64_t)(h - p.kv_heads) * p.vo_head
                          : p.k_out + token * p.ko_token + (int64_t)h * p.ko_head;
      *reinterpret_cast<u32x4*>(dst + 2 * d) = out;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int32_t kMaxRowDim = 512;   // a wave holds whole heads: 64 chunks of 8

inline int64_t row_bytes_of(int32_t format, int64_t dim) {
  return format == KVSTORE_FMT_FP4 ? dim / 2
         : format == KVSTORE_FMT_BF16 || format == KVSTORE_FMT_FP16 ? 2 * dim
                                                                    : dim;
}

// Largest byte offset that page and offset strides reach, plus `tail`, fits in
// int64 (strides >= 0).
bool paged_span_fits(int64_t num_slots, int64_t page_size, int64_t page, int64_t offset,
                     int64_t tail) {
  const int64_t max_page = (num_slots - 1) / page_size;
  const int64_t in_page = num_slots < page_size ? num_slots : page_size;
  return fits(max_page + 1, page) && fits(in_page, offset) &&
         sum_fits(max_page * page, in_page * offset, tail);
}

int check_paged_cache(const kvstore_paged_cache& c, bool reads_scales) {
  if (c.format < KVSTORE_FMT_BF16 || c.format > KVSTORE_FMT_FP4) return KVSTORE_ERR_DTYPE;
  const bool fp4 = c.format == KVSTORE_FMT_FP4;
  const bool fp8 = c.format == KVSTORE_FMT_E4M3FN || c.format == KVSTORE_FMT_E5M2;
  const bool kind_ok = fp4   ? c.scale_kind == KVSTORE_SCALES_BLOCK
                       : fp8 ? c.scale_kind >= KVSTORE_SCALES_TENSOR &&
                                   c.scale_kind <= KVSTORE_SCALES_TOKEN_HEAD
                             : c.scale_kind == KVSTORE_SCALES_TENSOR;
  if (!kind_ok) return KVSTORE_ERR_DTYPE;
  if (!c.k || !c.v) return KVSTORE_ERR_NULL;
  const bool per_slot = fp4 || (fp8 && c.scale_kind != KVSTORE_SCALES_TENSOR);
  if (per_slot && (!c.k_scales || !c.v_scales)) return KVSTORE_ERR_NULL;
  if (c.num_heads <= 0 || c.head_dim <= 0 || c.head_dim % (fp4 ? 32 : 16) ||
      c.head_dim > kMaxRowDim || c.page_size <= 0 || c.num_slots <= 0)
    return KVSTORE_ERR_SHAPE;
  const int64_t strides[6] = {c.k_stride_page, c.k_stride_offset, c.k_stride_head,
                              c.v_stride_page, c.v_stride_offset, c.v_stride_head};
  for (int64_t s : strides) {
    if (s < 0) return KVSTORE_ERR_SHAPE;
    if (!aligned(s, 16)) return KVSTORE_ERR_ALIGN;
  }
  const int64_t row = row_bytes_of(c.format, c.head_dim);
  if (!span_fits_int32(c.num_heads, c.k_stride_head, row) ||
      !span_fits_int32(c.num_heads, c.v_stride_head, row) ||
      !paged_span_fits(c.num_slots, c.page_size, c.k_stride_page, c.k_stride_offset, INT32_MAX) ||
      !paged_span_fits(c.num_slots, c.page_size, c.v_stride_page, c.v_stride_offset, INT32_MAX))
    return KVSTORE_ERR_SHAPE;
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return KVSTORE_ERR_ALIGN;
  if (per_slot) {
    const int64_t unit = fp4 ? 1 : 4;
    const int64_t ss[6] = {c.ks_stride_page, c.ks_stride_offset, c.ks_stride_head,
                           c.vs_stride_page, c.vs_stride_offset, c.vs_stride_head};
    for (int64_t s : ss) {
      if (s < 0) return KVSTORE_ERR_SHAPE;
      if (!aligned(s, unit)) return KVSTORE_ERR_ALIGN;
    }
    const int64_t tail = fp4 ? c.head_dim / 32 : 4;
    if (!span_fits_int32(c.num_heads, c.ks_stride_head, tail) ||
        !span_fits_int32(c.num_heads, c.vs_stride_head, tail) ||
        !paged_span_fits(c.num_slots, c.page_size, c.ks_stride_page, c.ks_stride_offset,
                         INT32_MAX) ||
        !paged_span_fits(c.num_slots, c.page_size, c.vs_stride_page, c.vs_stride_offset,
                         INT32_MAX))
      return KVSTORE_ERR_SHAPE;
    if (!aligned(c.k_scales, unit) || !aligned(c.v_scales, unit)) return KVSTORE_ERR_ALIGN;
  } else if (reads_scales && fp8) {
    if (!aligned(c.k_scales, 4) || !aligned(c.v_scales, 4)) return KVSTORE_ERR_ALIGN;
  }
  return KVSTORE_OK;
}

CacheSide cache_side(const kvstore_paged_cache& c, bool is_v) {
  CacheSide s;
  s.data = static_cast<uint8_t*>(is_v ? c.v : c.k);
  s.page = is_v ? c.v_stride_page : c.k_stride_page;
  s.offset = is_v ? c.v_stride_offset : c.k_stride_offset;
  s.head = is_v ? c.v_stride_head : c.k_stride_head;
  s.scales = static_cast<uint8_t*>(is_v ? c.v_scales : c.k_scales);
  s.s_page = is_v ? c.vs_stride_page : c.ks_stride_page;
  s.s_offset = is_v ? c.vs_stride_offset : c.ks_stride_offset;
  s.s_head = is_v ? c.vs_stride_head : c.ks_stride_head;
  return s;
}

int page_shift_of(int64_t page_size) {
  if (page_size & (page_size - 1)) return -1;
  int sh = 0;
  while ((int64_t(1) << sh) < page_size) ++sh;
  return sh;
}

// Row strides of [batch, heads, dim] 16-bit rows.
int check_row_strides(int64_t token, int64_t head, int64_t heads, int64_t dim, uint32_t batch) {
  if (token < 0 || head < 0) return KVSTORE_ERR_SHAPE;
  if (!aligned(token, 16) || !aligned(head, 16)) return KVSTORE_ERR_ALIGN;
  if (!span_fits_int32(heads, head, 2 * dim) || !fits((int64_t)batch + 1, token) ||
      !sum_fits((int64_t)batch * token, INT32_MAX, 0))
    return KVSTORE_ERR_SHAPE;
  return KVSTORE_OK;
}

void fill_rows(RowsParams& r, const kvstore_paged_cache& c, const void* indices, int idx_dtype,
               int64_t idx_stride) {
  r.k_side = cache_side(c, false);
  r.v_side = cache_side(c, true);
  r.indices = indices;
  r.idx_stride = idx_stride;
  r.idx64 = idx_dtype == KVSTORE_IDX_I64;
  r.num_slots = c.num_slots;
  r.page_size = c.page_size;
  r.page_shift = page_shift_of(c.page_size);
  r.chunks = (uint32_t)c.head_dim / 8;
  r.heads_per_wave = kWave / r.chunks;
}

// Heads per lane: four for long batches (their loads are in flight together
// and share the cosines), one where that would leave CUs without a wave.
// Appended tokens of 32 + 2 x 8 heads of 128 dims, one head a lane / four: 16
// tokens 3.3 / 4.6 us, 256 3.5 / 4.9, 1024 7.6 / 7.3, 4096 21.9 / 19.5, 16384
// 78.2 / 60.8; loaded tokens of 2 x 8: 1024 3.5 / 4.5, 4096 6.7 / 6.5, 16384
// 18.8 / 15.1.
constexpr int kRowsHeads = 4;
constexpr int64_t kRowsManyWaves = 2048;

// Groups of a token may not exceed this, so that every run holds a token.
constexpr int64_t kMaxRowGroups = int64_t(1) << 24;

// Calls fn(grid) for runs of tokens of at most 2^24 waves (2^30 work-items).
template <typename F>
int launch_rows(RowsParams& r, uint32_t batch, F&& fn) {
  const int64_t most = kMaxRowGroups * r.heads_per_wave / r.groups;
  for (uint32_t base = 0; base < batch;) {
    const int64_t left = batch - base, cap = most < kMaxLaunchTokens ? most : kMaxLaunchTokens;
    const uint32_t n = (uint32_t)(left < cap ? left : cap);
    r.token_base = base;
    r.batch = n;
    const int64_t waves = ceil_div((int64_t)n * r.groups, r.heads_per_wave);
    const int st = fn(dim3((uint32_t)ceil_div(waves, kRowsWaves)));
    if (st != KVSTORE_OK) return st;
    base += n;
  }
  return KVSTORE_OK;
}

template <bool kFp16, int kFmt, int kRope>
int launch_rope_heads(const RopeParams& p, int heads, dim3 grid, hipStream_t s) {
  const dim3 block(kWave * kRowsWaves);
  if (heads == 1) return launch(kvstore_rope_kernel<kFp16, kFmt, kRope, 1>, grid, block, 0, s, p);
  return launch(kvstore_rope_kernel<kFp16, kFmt, kRope, kRowsHeads>, grid, block, 0, s, p);
}

template <bool kFp16, int kFmt>
int launch_rope_kind(const RopeParams& p, int rope, int heads, dim3 grid, hipStream_t s) {
  switch (rope) {
    case kNoRope: return launch_rope_heads<kFp16, kFmt, kNoRope>(p, heads, grid, s);
    case kHalves: return launch_rope_heads<kFp16, kFmt, kHalves>(p, heads, grid, s);
    default: return launch_rope_heads<kFp16, kFmt, kInterleaved>(p, heads, grid, s);
  }
}

template <bool kFp16>
int launch_rope_fmt(const RopeParams& p, int fmt, int rope, int heads, dim3 grid, hipStream_t s) {
  switch (fmt) {
    case kRow16: return launch_rope_kind<kFp16, kRow16>(p, rope, heads, grid, s);
    case kRowE4M3: return launch_rope_kind<kFp16, kRowE4M3>(p, rope, heads, grid, s);
    case kRowE5M2: return launch_rope_kind<kFp16, kRowE5M2>(p, rope, heads, grid, s);
    default: return launch_rope_kind<kFp16, kRowFp4>(p, rope, heads, grid, s);
  }
}

template <bool kFp16, int kFmt>
int launch_load_heads(const LoadParams& p, int heads, dim3 grid, hipStream_t s) {
  const dim3 block(kWave * kRowsWaves);
  if (heads == 1) return launch(kvstore_load_kernel<kFp16, kFmt, 1>, grid, block, 0, s, p);
  return launch(kvstore_load_kernel<kFp16, kFmt, kRowsHeads>, grid, block, 0, s, p);
}

template <bool kFp16>
int launch_load_fmt(const LoadParams& p, int fmt, int heads, dim3 grid, hipStream_t s) {
  switch (fmt) {
    case kRow16: return launch_load_heads<kFp16, kRow16>(p, heads, grid, s);
    case kRowE4M3: return launch_load_heads<kFp16, kRowE4M3>(p, heads, grid, s);
    case kRowE5M2: return launch_load_heads<kFp16, kRowE5M2>(p, heads, grid, s);
    default: return launch_load_heads<kFp16, kRowFp4>(p, heads, grid, s);
  }
}

int row_fmt(int32_t format) {
  switch (format) {
    case KVSTORE_FMT_E4M3FN: return kRowE4M3;
    case KVSTORE_FMT_E5M2: return kRowE5M2;
    case KVSTORE_FMT_FP4: return kRowFp4;
    default: return kRow16;
  }
}

// Heads of a lane and groups of a token for `total` heads.
int set_rows_groups(RowsParams& r, int64_t total, uint32_t batch) {
  const int64_t waves = ceil_div((int64_t)batch * ceil_div(total, kRowsHeads), r.heads_per_wave);
  const int heads = waves >= kRowsManyWaves ? kRowsHeads : 1;
  r.groups = (uint32_t)ceil_div(total, heads);
  return heads;
}

bool fp16_format(int32_t format) { return format == KVSTORE_FMT_FP16; }

}  // namespace

extern "C" {

int kvstore_rope_paged(const kvstore_rope_rows* rows, const void* positions, int pos_dtype,
                       const float* cos_sin, int64_t cos_sin_stride, int64_t num_positions,
                       int32_t rot_dim, int interleaved, const void* indices, int idx_dtype,
                       int64_t idx_stride, const kvstore_paged_cache* cache,
                       const float* inv_k_scale_ptr, const float* inv_v_scale_ptr, uint32_t batch,
                       hipStream_t stream) {
  if (!rows || !cache) return KVSTORE_ERR_NULL;
  if (idx_dtype != KVSTORE_IDX_I32 && idx_dtype != KVSTORE_IDX_I64) return KVSTORE_ERR_DTYPE;
  if (pos_dtype != KVSTORE_IDX_I32 && pos_dtype != KVSTORE_IDX_I64) return KVSTORE_ERR_DTYPE;
  if (rows->src_dtype != KVSTORE_SRC_BF16 && rows->src_dtype != KVSTORE_SRC_FP16)
    return KVSTORE_ERR_DTYPE;
  if (batch == 0) return KVSTORE_OK;
  const kvstore_paged_cache& c = *cache;
  int st = check_paged_cache(c, false);
  if (st != KVSTORE_OK) return st;
  const bool fp16 = rows->src_dtype == KVSTORE_SRC_FP16;
  const int fmt = row_fmt(c.format);
  if (fmt == kRow16 && fp16_format(c.format) != fp16) return KVSTORE_ERR_DTYPE;
  if ((fmt == kRowE4M3 || fmt == kRowE5M2) && c.scale_kind != KVSTORE_SCALES_TENSOR)
    return KVSTORE_ERR_DTYPE;
  if (!rows->k || !rows->v || !indices || (rows->q && !rows->q_out) ||
      (cos_sin == nullptr) != (positions == nullptr))
    return KVSTORE_ERR_NULL;
  const int64_t dim = c.head_dim;
  int64_t q_heads = 0;
  if (rows->q) {
    q_heads = rows->q_heads;
    if (q_heads <= 0) return KVSTORE_ERR_SHAPE;
    st = check_row_strides(rows->q_stride_token, rows->q_stride_head, q_heads, dim, batch);
    if (st != KVSTORE_OK) return st;
    st = check_row_strides(rows->qo_stride_token, rows->qo_stride_head, q_heads, dim, batch);
    if (st != KVSTORE_OK) return st;
    if (!aligned(rows->q, 16) || !aligned(rows->q_out, 16)) return KVSTORE_ERR_ALIGN;
    if (rows->q == rows->q_out && (rows->q_stride_token != rows->qo_stride_token ||
                                   rows->q_stride_head != rows->qo_stride_head))
      return KVSTORE_ERR_SHAPE;
  }
  st = check_row_strides(rows->k_stride_token, rows->k_stride_head, c.num_heads, dim, batch);
  if (st != KVSTORE_OK) return st;
  st = check_row_strides(rows->v_stride_token, rows->v_stride_head, c.num_heads, dim, batch);
  if (st != KVSTORE_OK) return st;
  if (!aligned(rows->k, 16) || !aligned(rows->v, 16)) return KVSTORE_ERR_ALIGN;
  if (!aligned(inv_k_scale_ptr, 4) || !aligned(inv_v_scale_ptr, 4)) return KVSTORE_ERR_ALIGN;
  if (cos_sin) {
    if (rot_dim <= 0 || rot_dim % 16 || rot_dim > dim || num_positions <= 0 ||
        cos_sin_stride < 4 * (int64_t)rot_dim || !fits(num_positions, cos_sin_stride))
      return KVSTORE_ERR_SHAPE;
    if (!aligned(cos_sin, 16) || !aligned(cos_sin_stride, 16) ||
        !aligned(positions, pos_dtype == KVSTORE_IDX_I64 ? 8 : 4))
      return KVSTORE_ERR_ALIGN;
  }
  st = check_index_args(indices, idx_dtype, idx_stride, batch);
  if (st != KVSTORE_OK) return st;

  RopeParams p;
  fill_rows(p.rows, c, indices, idx_dtype, idx_stride);
  p.q = static_cast<const uint8_t*>(rows->q);
  p.k = static_cast<const uint8_t*>(rows->k);
  p.v = static_cast<const uint8_t*>(rows->v);
  p.q_out = static_cast<uint8_t*>(rows->q_out);
  p.q_token = rows->q_stride_token;
  p.q_head = rows->q_stride_head;
  p.qo_token = rows->qo_stride_token;
  p.qo_head = rows->qo_stride_head;
  p.k_token = rows->k_stride_token;
  p.k_head = rows->k_stride_head;
  p.v_token = rows->v_stride_token;
  p.v_head = rows->v_stride_head;
  p.positions = positions;
  p.cos_sin = reinterpret_cast<const uint8_t*>(cos_sin);
  p.cos_sin_stride = cos_sin_stride;
  p.num_positions = num_positions;
  p.inv_k = inv_k_scale_ptr;
  p.inv_v = inv_v_scale_ptr;
  p.q_heads = (uint32_t)q_heads;
  p.kv_heads = (uint32_t)c.num_heads;
  p.rot = cos_sin ? (uint32_t)rot_dim : 0;
  p.pos64 = pos_dtype == KVSTORE_IDX_I64;
  const int64_t total = q_heads + 2 * (int64_t)c.num_heads;
  if (total > kMaxRowGroups) return KVSTORE_ERR_SHAPE;
  const int heads = set_rows_groups(p.rows, total, batch);
  const int rope = !cos_sin ? kNoRope : interleaved ? kInterleaved : kHalves;
  return launch_rows(p.rows, batch, [&](dim3 grid) {
    return fp16 ? launch_rope_fmt<true>(p, fmt, rope, heads, grid, stream)
                : launch_rope_fmt<false>(p, fmt, rope, heads, grid, stream);
  });
}

int kvstore_load_paged(const kvstore_paged_cache* cache, const void* indices, int idx_dtype,
                       int64_t idx_stride, void* k_out, int64_t ko_stride_token,
                       int64_t ko_stride_head, void* v_out, int64_t vo_stride_token,
                       int64_t vo_stride_head, int dst_dtype, uint32_t batch, hipStream_t stream) {
  if (!cache) return KVSTORE_ERR_NULL;
  if (idx_dtype != KVSTORE_IDX_I32 && idx_dtype != KVSTORE_IDX_I64) return KVSTORE_ERR_DTYPE;
  if (dst_dtype != KVSTORE_SRC_BF16 && dst_dtype != KVSTORE_SRC_FP16) return KVSTORE_ERR_DTYPE;
  if (batch == 0) return KVSTORE_OK;
  const kvstore_paged_cache& c = *cache;
  int st = check_paged_cache(c, true);
  if (st != KVSTORE_OK) return st;
  const bool fp16 = dst_dtype == KVSTORE_SRC_FP16;
  const int fmt = row_fmt(c.format);
  if (fmt == kRow16 && fp16_format(c.format) != fp16) return KVSTORE_ERR_DTYPE;
  if (!indices || !k_out || !v_out) return KVSTORE_ERR_NULL;
  st = check_row_strides(ko_stride_token, ko_stride_head, c.num_heads, c.head_dim, batch);
  if (st != KVSTORE_OK) return st;
  st = check_row_strides(vo_stride_token, vo_stride_head, c.num_heads, c.head_dim, batch);
  if (st != KVSTORE_OK) return st;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return KVSTORE_ERR_ALIGN;
  st = check_index_args(indices, idx_dtype, idx_stride, batch);
  if (st != KVSTORE_OK) return st;
  const int64_t total = 2 * (int64_t)c.num_heads;
  if (total > kMaxRowGroups) return KVSTORE_ERR_SHAPE;

  LoadParams p;
  fill_rows(p.rows, c, indices, idx_dtype, idx_stride);
  p.k_out = static_cast<uint8_t*>(k_out);
  p.v_out = static_cast<uint8_t*>(v_out);
  p.ko_token = ko_stride_token;
  p.ko_head = ko_stride_head;
  p.vo_token = vo_stride_token;
  p.vo_head = vo_stride_head;
  p.k_scale = static_cast<const float*>(c.k_scales);
  p.v_scale = static_cast<const float*>(c.v_scales);
  p.kv_heads = (uint32_t)c.num_heads;
  p.scale_kind = c.scale_kind;
  const int heads = set_rows_groups(p.rows, total, batch);
  return launch_rows(p.rows, batch, [&](dim3 grid) {
    return fp16 ? launch_load_fmt<true>(p, fmt, heads, grid, stream)
                : launch_load_fmt<false>(p, fmt, heads, grid, stream);
  });
}

}  // extern "C"
