// Paged attention for few rows (up to 16 of a sequence and kv head): compiled once
// per source type and cache format (KVATTN_FP16, KVATTN_FMT).
//
//   out = sum_k softmax_k(c q . K_k) V_k over the keys that a row sees.
//
// A block owns a tile of up to 16 rows (tokens x q heads of one kv head) and one
// split of its keys.  Its four waves take the split's 32-key steps in turn, each
// with a running maximum and sum of its own, and are joined through LDS at the
// end; splits are joined by kvattn_join_kernel.
//
// Per step, S^T = K Q^T on 16x16x32 MFMAs: a K row's lanes load straight from
// the cache into the operand's registers (the dims of a dot product may come in
// any order, so a lane loads 16 consecutive bytes whatever the format).  S^T
// leaves a lane with four consecutive keys of one row, which is how the second
// product, O^T = V^T P^T, wants P^T once the keys of the two 16-key halves are
// interleaved; V goes through LDS and is read back transposed, four keys of a
// column at a time.  Nothing but V passes through LDS, and no wave waits for
// another inside the loop.
//
// The running maximum is raised only when a score exceeds it by more than 2^8:
// until then weights stay below 2^8, exact enough in fp32 sums and in range in
// either 16-bit type, and most steps skip the cross-lane maximum and the
// rescaling of O.
//
// Bound by the latency of loads and the work of a step together: 32 contexts of
// up to 32768 4-bit keys (32 q heads on 8 of 128 dims, 591 MB) take 157 us, 3.8
// TB/s, and 102 us when all pages are the same few, in cache; 64 windows of 4096
// e4m3fn keys (452 MB) 106 us, 4.3 TB/s, and 71 us.  One sequence of 777 bf16 keys
// takes 10.4 us, two launches of serial latencies.
#include "attention_device.h"
#include "kvstore.h"

namespace kvattn {
namespace {

constexpr int kWaves = 4;
constexpr bool kFp16 = KVATTN_FP16 != 0;
constexpr int kFmt = KVATTN_FMT;
constexpr bool kFp8 = kFmt == kFmtE4M3 || kFmt == kFmtE5M2;
constexpr float kLazy = 8.0f;
constexpr int kStep = kSplitStep;

// Bytes that d elements take.
__device__ __forceinline__ uint32_t bytes_of(int32_t d) {
  return kFmt == kFmt16 ? 2 * d : kFmt == kFmtFp4 ? d / 2 : d;
}

template <int kDim>
struct Shape {
  // Blocks of 8 elements that a lane loads of a K row at a time.
  static constexpr int kEB = kFmt == kFmt16 ? 1 : kFmt == kFmtFp4 && kDim >= 128 ? 4 : 2;
  static constexpr int kLoadsK = kDim / 32 / kEB;
  // A lane loads 16 bytes of a V row at a time.
  static constexpr int kVE = kFmt == kFmt16 ? 8 : kFmt == kFmtFp4 ? 32 : 16;
  static constexpr int kLanesV = kDim / kVE;            // lanes per V row
  static constexpr int kRowsV = 64 / kLanesV;           // V rows per access
  static constexpr int kLoadsV = kStep / kRowsV;
  static constexpr int kStrideV = 2 * kDim + 32;        // bytes of a V row in LDS
  static constexpr int kStrideO = kDim + 4;             // floats of an O row in LDS
};

// A lane's piece of a K row: 16 bytes, or 8 of a 4-bit row of up to 64 dims.
template <int kBytes>
__device__ __forceinline__ void load_piece(uint64_t at, u32x4* x) {
  if constexpr (kBytes == 16) {
    *x = load_global<u32x4>(at);
  } else {
    const u32x2 y = load_global<u32x2>(at);
    *x = u32x4{y.x, y.y, 0u, 0u};
  }
}

template <int kDim, bool kWholePages>
struct WaveLds {
  alignas(16) uint8_t v[kStep * Shape<kDim>::kStrideV];
  alignas(16) float scale[2][kFp8 ? kStep : 4];
  // addresses of the step's K and V rows
  uint64_t at[2][kWholePages ? 1 : kStep];
  uint64_t scale_at[2][kFmt == kFmtFp4 && !kWholePages ? kStep : 1];
};

__device__ __forceinline__ float group_max4(float x) {   // over the 4 lanes l, l^16, l^32, l^48
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}

__device__ __forceinline__ uint32_t load_scalar(const int32_t* p) {
  return *reinterpret_cast<__attribute__((address_space(4))) const uint32_t*>(
      reinterpret_cast<uint64_t>(p));
}

// kWholePages: page_size is a multiple of 16, so that the 16 keys of a half step
// lie in one page: their rows have a scalar base and fixed lane offsets, and
// page table reads are scalar loads.  Otherwise lanes look their keys' pages up
// and hand the addresses over through LDS.  kFull: the head has kDim dims.
template <int kDim, bool kWholePages, bool kFull>
__global__ __launch_bounds__(64 * kWaves, kDim <= 128 ? 3 : 1) void kvattn_split_kernel(
    const Params p) {
  typedef Shape<kDim> S;
  constexpr int kKs = kDim / 32;     // k steps of Q K^T
  constexpr int kDt = kDim / 16;     // column tiles of O
  __shared__ WaveLds<kDim, kWholePages> lds[kWaves];
  __shared__ float s_m[kWaves][kSplitRows], s_l[kWaves][kSplitRows];

  // Blocks go to the eight XCDs in turn.  The heads of one tile and split take
  // eight block numbers apart, so one XCD, which read the same cache lines where
  // a head's row is shorter than one (and the scales of all heads).
  const uint32_t turn = blockIdx.x >> 3, head = turn % p.kv_heads;
  // A tile's splits go to different XCDs, and one split's number to all of them
  // over the tiles: long sequences have more splits than others.
  const uint32_t eight = turn / p.kv_heads;
  const uint32_t unit = eight * 8 + ((blockIdx.x + eight + (eight >> 3)) & 7);
  const uint32_t slot = unit / p.splits, split = unit - slot * p.splits;
  if (slot >= p.tile_slots) return;
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const uint32_t g = lane >> 4, c16 = lane & 15;
  Tile<kStep> t;
  if (!tile_of(p, slot, kSplitRows, &t)) return;
  int32_t n_splits;
  const int32_t chunk = split_steps(p, t, &n_splits);
  if ((int32_t)split >= n_splits) return;
  const int32_t s_begin = split * chunk;
  const int32_t s_end = min(t.steps, s_begin + chunk);
  WaveLds<kDim, kWholePages>& my = lds[w];
  const int32_t dim = kFull ? kDim : p.dim;

  const bool dyn = kFp8 && p.scale_kind != KVATTN_TENSOR;
  float c = p.scale2, v_scale = 1.0f;
  if (kFp8 && !dyn) {
    if (p.k.scales) c *= *reinterpret_cast<const float*>(p.k.scales);
    if (p.v.scales) v_scale = *reinterpret_cast<const float*>(p.v.scales);
  }

  // Q^T operands and the positions of this lane's rows.
  u32x4 q[kKs];
  int32_t pos;
  {
    const int32_t row = t.row0 + ((int32_t)c16 < t.rows ? (int32_t)c16 : t.rows - 1);
    const int32_t tok = row / (int32_t)p.group;
    pos = t.first_pos + tok;
    const uint8_t* src = p.q + (int64_t)(t.token0 + tok) * p.q_token +
                         (int64_t)(head * p.group + (row - tok * (int32_t)p.group)) * p.q_head;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks) {
      const int d = (ks / S::kEB) * 32 * S::kEB + g * 8 * S::kEB + (ks % S::kEB) * 8;
      q[ks] = u32x4{0u, 0u, 0u, 0u};
      if (d < dim) q[ks] = *reinterpret_cast<const u32x4*>(src + 2 * d);
    }
  }

  f32x4 acc[kDt];
  float m = kNegInf, l = 0.0f;
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt) acc[dt] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int32_t* table = p.table + (int64_t)t.seq * p.table_stride;
  const int64_t head_k = (int64_t)head * p.k.head, head_v = (int64_t)head * p.v.head;
  const uint64_t k_from = reinterpret_cast<uint64_t>(p.k.data) + head_k;
  const uint64_t v_from_head = reinterpret_cast<uint64_t>(p.v.data) + head_v;
  const bool head_scales = kFmt == kFmtFp4 || p.scale_kind == KVATTN_TOKEN_HEAD;
  const uint64_t ks_from = reinterpret_cast<uint64_t>(p.k.scales) + (head_scales ? (int64_t)head * p.k.s_head : 0);
  const uint64_t vs_from = reinterpret_cast<uint64_t>(p.v.scales) + (head_scales ? (int64_t)head * p.v.s_head : 0);
  bool met_bad = false;

  // Keys of a step that some row of the tile may see, as bits.
  auto wanted = [&](int32_t key0) -> uint32_t {
    const uint32_t in = (uint32_t)low_bits(t.end - key0);
    return in & (~(uint32_t)low_bits(t.low - key0) | (uint32_t)low_bits(p.sinks < key0 ? 0 : p.sinks - key0));
  };

  // The pages of a step: of its halves (scalar), or of the lane's key lane & 31
  // (-2: no row of the tile sees it).
  struct Pages { int32_t a, b; };
  auto pages_of = [&](int32_t step) -> Pages {
    const int32_t key0 = t.key_of(step);
    int32_t page, off;
    if constexpr (kWholePages) {
      const int32_t last = (t.end - 1) & ~15;   // a half without keys looks up the last one with some
      const int32_t ka = min(key0, last), kb = min(key0 + 16, last);
      key_page(p, ka, &page, &off);
      const int32_t a = load_scalar(table + page);
      key_page(p, kb, &page, &off);
      return {a, (int32_t)load_scalar(table + page)};
    } else {
      const int32_t kk = lane & 31;
      if (!((wanted(key0) >> kk) & 1u)) return {-2, -2};
      key_page(p, key0 + kk, &page, &off);
      return {table[page], 0};
    }
  };

  u32x4 kr[2][S::kLoadsK], vr[S::kLoadsV];
  uint32_t kb[2][kFmt == kFmtFp4 ? S::kLoadsK : 1], vb[kFmt == kFmtFp4 ? S::kLoadsV : 1];
  float sc = 1.0f;     // K's (lanes 0-31) or V's scale of key lane & 31, whether that is there or not
  uint32_t ok = 0;     // the step's keys that are there

  // Lanes past the head's dims load a row's start, and write or multiply nothing.
  const int32_t dk = g * 8 * S::kEB;
  const int32_t v_row = lane / S::kLanesV, dv = (lane % S::kLanesV) * S::kVE;
  const bool writes = dv < dim;
  const uint32_t v_from = writes ? bytes_of(dv) : 0;

  // Places the step's keys and issues their loads.
  auto load_step = [&](int32_t step, Pages pg) {
    const int32_t key0 = t.key_of(step);
    const uint32_t want = wanted(key0);
    if constexpr (kWholePages) {
      const bool ga = (uint32_t)pg.a < (uint32_t)p.num_pages, gb = (uint32_t)pg.b < (uint32_t)p.num_pages;
      const uint32_t there = (ga ? 0xFFFFu : 0u) | (gb ? 0xFFFF0000u : 0u);
      met_bad = met_bad || (want & ~there) != 0;
      ok = want & there;
      // page 0 stands in for a page that is not there
      const uint32_t page[2] = {ga ? (uint32_t)pg.a : 0u, gb ? (uint32_t)pg.b : 0u};
      int32_t ignore, off[2];
      key_page(p, key0, &ignore, &off[0]);
      key_page(p, key0 + 16, &ignore, &off[1]);
      // strides are below 2^32 here (the launch sees to it)
      uint64_t kbase[2], vbase[2], ksbase[2], vsbase[2];
      auto base_of = [&](uint64_t from, int64_t page_stride, int64_t stride, int h) {
        return from + (uint64_t)page[h] * (uint32_t)page_stride + (uint64_t)(uint32_t)off[h] * (uint32_t)stride;
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        kbase[h] = base_of(k_from, p.k.page, p.k.offset, h);
        vbase[h] = base_of(v_from_head, p.v.page, p.v.offset, h);
        if (kFmt == kFmtFp4 || dyn) {
          ksbase[h] = base_of(ks_from, p.k.s_page, p.k.s_offset, h);
          vsbase[h] = base_of(vs_from, p.v.s_page, p.v.s_offset, h);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < S::kLoadsK; ++i) {
          const int32_t d = dk + i * 32 * S::kEB;
          const uint32_t from = c16 * (uint32_t)p.k.offset + (d < dim ? bytes_of(d) : 0);
          load_piece<kFmt == kFmtFp4 ? 4 * S::kEB : 16>(kbase[h] + from, &kr[h][i]);
          if constexpr (kFmt == kFmtFp4)
            kb[h][i] = load_global<uint8_t>(ksbase[h] + (uint32_t)(c16 * (uint32_t)p.k.s_offset + (d < dim ? d / 32 : 0)));
        }
#pragma unroll
      for (int i = 0; i < S::kLoadsV; ++i) {
        uint64_t base, sbase;
        uint32_t row;
        if constexpr (S::kRowsV > 16) {   // both halves in one access
          base = lane < 32 ? vbase[0] : vbase[1];
          sbase = lane < 32 ? vsbase[0] : vsbase[1];
          row = v_row & 15;
        } else {
          constexpr int per = 16 / (S::kRowsV > 16 ? 16 : S::kRowsV);
          base = vbase[i / per] + (i % per) * S::kRowsV * p.v.offset;
          sbase = vsbase[i / per] + (i % per) * S::kRowsV * p.v.s_offset;
          row = v_row;
        }
        vr[i] = load_global<u32x4>(base + (uint32_t)(row * (uint32_t)p.v.offset + v_from));
        if constexpr (kFmt == kFmtFp4)
          vb[i] = load_global<uint8_t>(sbase + (uint32_t)(row * (uint32_t)p.v.s_offset + (writes ? dv / 32 : 0)));
      }
      if constexpr (kFp8) {
        if (dyn) {
          const uint64_t base = lane < 32 ? (lane < 16 ? ksbase[0] : ksbase[1]) : (lane < 48 ? vsbase[0] : vsbase[1]);
          sc = load_global<float>(base + (int64_t)c16 * (lane < 32 ? p.k.s_offset : p.v.s_offset));
        }
      }
    } else {
      const int32_t kk = lane & 31;
      int32_t ignore, off;
      key_page(p, key0 + kk, &ignore, &off);
      const bool there = pg.a >= 0 && pg.a < p.num_pages;
      met_bad = met_bad || (pg.a != -2 && !there);
      ok = (uint32_t)__ballot(there);
      // slot 0 stands in for keys that are not there
      const int64_t page = there ? pg.a : 0, of = there ? off : 0;
      const Side& side = lane < 32 ? p.k : p.v;
      my.at[lane >> 5][kk] = reinterpret_cast<uint64_t>(side.data) + page * side.page + of * side.offset +
                             (lane < 32 ? head_k : head_v);
      const uint64_t scales = reinterpret_cast<uint64_t>(side.scales) + page * side.s_page + of * side.s_offset;
      if constexpr (kFmt == kFmtFp4) my.scale_at[lane >> 5][kk] = scales + (int64_t)head * side.s_head;
      if constexpr (kFp8) {
        if (dyn)
          sc = load_global<float>(scales + (p.scale_kind == KVATTN_TOKEN_HEAD ? (int64_t)head * side.s_head : 0));
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < S::kLoadsK; ++i) {
          const int32_t d = dk + i * 32 * S::kEB;
          load_piece<kFmt == kFmtFp4 ? 4 * S::kEB : 16>(
              my.at[0][h * 16 + c16] + (d < dim ? bytes_of(d) : 0), &kr[h][i]);
          if constexpr (kFmt == kFmtFp4)
            kb[h][i] = load_global<uint8_t>(my.scale_at[0][h * 16 + c16] + (d < dim ? d / 32 : 0));
        }
#pragma unroll
      for (int i = 0; i < S::kLoadsV; ++i) {
        const int row = i * S::kRowsV + v_row;
        vr[i] = load_global<u32x4>(my.at[1][row] + v_from);
        if constexpr (kFmt == kFmtFp4) vb[i] = load_global<uint8_t>(my.scale_at[1][row] + (writes ? dv / 32 : 0));
      }
      __builtin_amdgcn_wave_barrier();
    }
  };

  // Where rows see different keys, NaN and infinities of V (0 * V is not 0 for
  // them) are left out of the product, and added at the end to the rows that do
  // see them.
  const bool ragged = t.p_lo != t.p_hi;
  bool special = false;
  auto mixed_step = [&](int32_t key0) {   // some row does not see some key
    return ok != 0xFFFFFFFFu || key0 + kStep - 1 > t.p_lo ||
           !(t.p_hi - key0 < p.window || key0 + kStep - 1 < p.sinks);
  };

  // V of the step into LDS as 16-bit values.
  auto store_v = [&](bool mixed) {
    const bool clean = ragged && mixed;
#pragma unroll
    for (int i = 0; i < S::kLoadsV; ++i) {
      const int row = i * S::kRowsV + v_row;
      u32x4 x = vr[i];
      uint32_t byte = kFmt == kFmtFp4 ? vb[kFmt == kFmtFp4 ? i : 0] : 0;
      if (mixed) {   // 0 * V must be 0 for keys that are not there
        const bool there = (ok >> row) & 1u;
        x = there ? x : u32x4{0u, 0u, 0u, 0u};
        byte = there ? byte : 127u;
      }
      uint8_t* dst = my.v + row * S::kStrideV + 2 * dv;
      if constexpr (kFmt == kFmt16) {
        if (clean) x = finite8<kFp16>(x, &special);
        if (writes) *reinterpret_cast<u32x4*>(dst) = x;
      } else if constexpr (kFmt == kFmtFp4) {
        if (clean && byte == 255) {
          special = true;
          byte = 127;
          x = u32x4{0u, 0u, 0u, 0u};
        }
        const float s4 = __uint_as_float(byte << 23);
        const uint32_t e4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (writes) *reinterpret_cast<u32x4*>(dst + 16 * e) = values8<kFp16, kFmt>(e4[e], 0, s4);
      } else {
        // The scale's power of two goes into the values, exactly; its
        // significand into the weights.
        const float s8 = dyn ? my.scale[1][row] : 1.0f;
        u32x4 y = values8<kFp16, kFmt>(x.x, x.y, s8), z = values8<kFp16, kFmt>(x.z, x.w, s8);
        if (clean) {
          y = finite8<kFp16>(y, &special);
          z = finite8<kFp16>(z, &special);
        }
        if (writes) {
          *reinterpret_cast<u32x4*>(dst) = y;
          *reinterpret_cast<u32x4*>(dst + 16) = z;
        }
      }
    }
  };

  if (!kFull) {   // the columns that no lane writes
    for (uint32_t i = lane; i < sizeof(my.v) / 16; i += 64)
      reinterpret_cast<u32x4*>(my.v)[i] = u32x4{0u, 0u, 0u, 0u};
  }

  int32_t step = s_begin + (int32_t)w;
  Pages next = {-2, -2};
  if (step < s_end) {
    load_step(step, pages_of(step));
    next = pages_of(min(step + kWaves, s_end - 1));
  }
  for (; step < s_end; step += kWaves) {
    const int32_t key0 = t.key_of(step);
    const uint32_t ok_now = ok;
    const bool mixed = mixed_step(key0);
    if constexpr (kFp8) {
      if (dyn) my.scale[lane >> 5][lane & 31] = (ok_now >> (lane & 31)) & 1u ? sc : 1.0f;
      __builtin_amdgcn_wave_barrier();
    }
    store_v(mixed);

    // S^T, in 16-key halves.
    f32x4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      s[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 raw = kr[h][ks / S::kEB];
        constexpr int kEB = S::kEB;
        const int e = ks % kEB;
        u32x4 a;
        if constexpr (kFmt == kFmt16) {
          a = raw;
        } else if constexpr (kFmt == kFmtFp4) {
          const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
          a = values8<kFp16, kFmt>(x[e], 0, __uint_as_float(kb[h][ks / kEB] << 23));
        } else {
          a = e ? values8<kFp16, kFmt>(raw.z, raw.w, 1.0f) : values8<kFp16, kFmt>(raw.x, raw.y, 1.0f);
        }
        // q is 0 past the head's dims; what was loaded in their place need not be finite
        if (!kFull && dk + (ks / kEB) * 32 * kEB + e * 8 >= dim) a = u32x4{0u, 0u, 0u, 0u};
        s[h] = mfma16<kFp16>(a, q[ks], s[h]);
      }
    }

    // Scales of the lane's keys: 4g ... 4g + 3 of each half.
    f32x4 ksc[2], vsc[2];
    if constexpr (kFp8) {
      if (dyn) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ksc[h] = *reinterpret_cast<const f32x4*>(&my.scale[0][h * 16 + 4 * g]);
          vsc[h] = *reinterpret_cast<const f32x4*>(&my.scale[1][h * 16 + 4 * g]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            vsc[h][i] = __uint_as_float((__float_as_uint(vsc[h][i]) & 0x807FFFFFu) | 0x3F800000u);
        }
      }
    }

    // The next step's loads fly during the rest of this one.
    if (step + kWaves < s_end) {
      load_step(step + kWaves, next);
      next = pages_of(min(step + 2 * kWaves, s_end - 1));
    }

    float x[8];
    float top = kNegInf;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[4 * h + i] = s[h][i] * (dyn ? c * ksc[h][i] : c);
    uint32_t seen = ~0u;   // bits i and 16 + i: the row sees the lane's key i of half 0 and 1
    if (mixed) {
      seen = (uint32_t)seen_bits(p, pos, key0, ok_now) >> (4 * g);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = seen & (1u << ((i >> 2) * 16 + (i & 3))) ? x[i] : kNegInf;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, x[i]);
    if (__ballot(top > m + kLazy || (m == kNegInf && top > kNegInf)) != 0) {
      const float was = m, now = fmaxf(was, group_max4(top));
      const float f = now == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(was - now);
      m = now;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[dt][i] *= f;
    }
    const float base = m == kNegInf ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = __builtin_amdgcn_exp2f(x[i] - base);
      l += x[i];
    }
    if (dyn) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = x[i] * vsc[i >> 2][i & 3];
        x[i] = seen & (1u << ((i >> 2) * 16 + (i & 3))) ? y : 0.0f;
      }
    }
    const u32x4 pt =    // P^T operand
        u32x4{pack_pair<kFp16>(x[0], x[1]), pack_pair<kFp16>(x[2], x[3]),
              pack_pair<kFp16>(x[4], x[5]), pack_pair<kFp16>(x[6], x[7])};

    // O^T += V^T P^T.
    __builtin_amdgcn_wave_barrier();
    uint8_t* const col = my.v + (4 * g + (c16 >> 2)) * S::kStrideV + (c16 & 3) * 8;
#pragma unroll
    for (int dt = 0; dt < kDt; ++dt) {
      const u32x2 a = read_column4(col + dt * 32);
      const u32x2 b = read_column4(col + 16 * S::kStrideV + dt * 32);
      const u32x4 vt = u32x4{a.x, a.y, b.x, b.y};
      acc[dt] = mfma16<kFp16>(vt, pt, acc[dt]);
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (__ballot(met_bad) != 0 && head == 0 && lane == 0)
    report(p.flag, (uint32_t)(t.token0 + t.row0 / (int32_t)p.group));

  if (__ballot(special) != 0) {
    // Rare: V's NaN and infinities of the steps that they were left out of, for
    // the rows that see them.
    for (step = s_begin + (int32_t)w; step < s_end; step += kWaves) {
      const int32_t first = t.key_of(step);
      for (int32_t key = first; key < min(first + kStep, t.end); ++key) {
        if (key < t.low && key >= p.sinks) continue;
        int32_t page, off;
        key_page(p, key, &page, &off);
        page = table[page];
        if (page < 0 || page >= p.num_pages) continue;
        int32_t d0 = 4 * g;
        asm volatile("" : "+v"(d0));
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (d0 + dt * 16 + i >= dim) continue;
            const float x = special_at<kFmt, kFp16>(p, head, page, off, d0 + dt * 16 + i);
            acc[dt][i] += sees(p, pos, key) ? x : 0.0f;
          }
      }
    }
  }

  // Join the waves.
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    s_m[w][c16] = m;
    s_l[w][c16] = l;
  }
  __syncthreads();
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) top = fmaxf(top, s_m[i][c16]);
  const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
  float* o = reinterpret_cast<float*>(my.v) + c16 * S::kStrideO + 4 * g;
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt) {
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = acc[dt][i] * f;
    *reinterpret_cast<f32x4*>(o + dt * 16) = y;
  }
  __syncthreads();
  // 16 threads per row, four columns at a time
  const int r = threadIdx.x >> 4, part = threadIdx.x & 15;
  if (r < t.rows) {
    float row_top = kNegInf, row_l = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) row_top = fmaxf(row_top, s_m[i][r]);
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const float mi = s_m[i][r];
      row_l += mi == kNegInf ? 0.0f : s_l[i][r] * __builtin_amdgcn_exp2f(mi - row_top);
    }
    const Row x = row_of(p, t, head, r);
    const int64_t at = x.index * p.splits + split;
    const float inv = row_l == 0.0f ? 0.0f : v_scale / row_l;
#pragma unroll
    for (int d = part * 4; d < kDim; d += 64) {
      f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kWaves; ++i)
        y += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds[i].v) +
                                             r * S::kStrideO + d);
      if (d >= dim) continue;
      if (n_splits == 1) {
        *reinterpret_cast<u32x2*>(p.out + x.token * p.o_token + (int64_t)x.head * p.o_head + 2 * d) =
            u32x2{pack_pair<kFp16>(y[0] * inv, y[1] * inv), pack_pair<kFp16>(y[2] * inv, y[3] * inv)};
      } else {
        *reinterpret_cast<f32x4*>(p.ws_o + at * dim + d) = y;
      }
    }
    if (n_splits > 1 && part == 0) {
      p.ws_ml[2 * at] = row_top;
      p.ws_ml[2 * at + 1] = row_l;
    }
  }
}

__global__ __launch_bounds__(256) void kvattn_join_kernel(const Params p) {
  join_splits<kFp16, kStep>(p, kSplitRows, kFp8 && p.scale_kind == KVATTN_TENSOR && p.v.scales
                                               ? *reinterpret_cast<const float*>(p.v.scales)
                                               : 1.0f);
}

int run(void (*kernel)(Params), dim3 grid, const Params& p, hipStream_t stream) {
  Params copy = p;
  void* argv[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(256), argv, 0, stream) ==
                 hipSuccess
             ? KVSTORE_OK
             : KVSTORE_ERR_HIP;
}

template <bool kWholePages, bool kFull>
int launch_dims(const Params& p, int padded_dim, hipStream_t stream) {
  const dim3 grid((p.tile_slots * p.splits + 7) / 8 * 8 * p.kv_heads);
  void (*kernel)(Params) = padded_dim == 64    ? kvattn_split_kernel<64, kWholePages, kFull>
                           : padded_dim == 128 ? kvattn_split_kernel<128, kWholePages, kFull>
                                               : kvattn_split_kernel<256, kWholePages, kFull>;
  const int st = run(kernel, grid, p, stream);
  if (st != KVSTORE_OK || p.splits == 1) return st;
  return run(kvattn_join_kernel, dim3(p.tile_slots * p.kv_heads * p.join_parts), p, stream);
}

}  // namespace

#define KVATTN_NAME2(src, fmt) launch_split_##src##_##fmt
#define KVATTN_NAME(src, fmt) KVATTN_NAME2(src, fmt)
#if KVATTN_FP16
#define KVATTN_SRC fp16
#else
#define KVATTN_SRC bf16
#endif

int KVATTN_NAME(KVATTN_SRC, KVATTN_FMT)(const Params& p, int padded_dim, hipStream_t stream) {
  // Whole pages: 32-bit strides, and 32-bit offsets of lanes into 16 rows.
  const int64_t most = INT32_MAX / 32;
  const bool whole = p.page_size % 16 == 0 && p.k.offset <= most && p.v.offset <= most &&
                     p.k.s_offset <= most && p.v.s_offset <= most && p.k.page <= INT32_MAX &&
                     p.v.page <= INT32_MAX && p.k.s_page <= INT32_MAX && p.v.s_page <= INT32_MAX;
  if (!whole) return launch_dims<false, false>(p, padded_dim, stream);
  return p.dim == padded_dim ? launch_dims<true, true>(p, padded_dim, stream)
                             : launch_dims<true, false>(p, padded_dim, stream);
}

}  // namespace kvattn
