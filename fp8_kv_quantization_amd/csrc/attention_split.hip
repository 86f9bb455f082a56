// Paged attention for few rows (single tokens, short runs, and chunks of long
// ones): compiled once per source type and cache format (KVATTN_FP16, KVATTN_FMT).
//
//   out = sum_k softmax_k(c q . K_k) V_k over the keys that a row sees.
//
// A block owns a tile of up to 16 * kNr rows (tokens x q heads of one kv head)
// and one split of its keys.  Its four waves take the split's 32-key steps in
// turn, each with a running maximum and sum of its own, and are joined through
// LDS at the end; splits are joined by kvattn_join_kernel.
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
#include "attention_device.h"
#include "kvstore.h"

namespace kvattn {
namespace {

constexpr int kWaves = 4;
constexpr bool kFp16 = KVATTN_FP16 != 0;
constexpr int kFmt = KVATTN_FMT;
constexpr float kLazy = 8.0f;
constexpr int kStep = kSplitStep;

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

template <int kDim>
struct WaveLds {
  alignas(16) uint8_t v[kStep * Shape<kDim>::kStrideV];
  int64_t at[2][kStep];      // K and V offsets of the step's keys, -1: not loaded
  int64_t scale_at[2][kFmt == kFmtFp4 ? kStep : 1];
  alignas(16) float scale[2][kFmt == kFmtE4M3 || kFmt == kFmtE5M2 ? kStep : 4];
};

__device__ __forceinline__ float group_max4(float x) {   // over the 4 lanes l, l^16, l^32, l^48
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}

template <int kDim, int kNr>
__global__ __launch_bounds__(64 * kWaves) void kvattn_split_kernel(const Params p) {
  typedef Shape<kDim> S;
  constexpr int kTileRows = 16 * kNr;
  constexpr int kKs = kDim / 32;     // k steps of Q K^T
  constexpr int kDt = kDim / 16;     // column tiles of O
  __shared__ WaveLds<kDim> lds[kWaves];
  __shared__ float s_m[kWaves][kTileRows], s_l[kWaves][kTileRows];

  const uint32_t head = blockIdx.x % p.kv_heads, slot = blockIdx.x / p.kv_heads;
  const uint32_t lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t g = lane >> 4, c16 = lane & 15;
  Tile<kStep> t;
  if (!tile_of(p, slot, kTileRows, &t)) return;
  int32_t n_splits;
  const int32_t chunk = split_steps(p, t, &n_splits);
  if ((int32_t)blockIdx.y >= n_splits) return;
  const int32_t s_begin = blockIdx.y * chunk;
  const int32_t s_end = min(t.steps, s_begin + chunk);
  WaveLds<kDim>& my = lds[w];

  const bool dyn = (kFmt == kFmtE4M3 || kFmt == kFmtE5M2) && p.scale_kind != KVATTN_TENSOR;
  const bool tensor = (kFmt == kFmtE4M3 || kFmt == kFmtE5M2) && p.scale_kind == KVATTN_TENSOR;
  float c = p.scale2, v_scale = 1.0f;
  if (tensor) {
    if (p.k.scales) c *= *reinterpret_cast<const float*>(p.k.scales);
    if (p.v.scales) v_scale = *reinterpret_cast<const float*>(p.v.scales);
  }

  // Q^T operands and the positions of this lane's rows.
  u32x4 q[kNr][kKs];
  int32_t pos[kNr];
#pragma unroll
  for (int n = 0; n < kNr; ++n) {
    const int32_t r = n * 16 + c16;
    const int32_t row = t.row0 + (r < t.rows ? r : t.rows - 1);
    const int32_t tok = row / (int32_t)p.group;
    pos[n] = t.first_pos + tok;
    const uint8_t* src = p.q + (int64_t)(t.token0 + tok) * p.q_token +
                         (int64_t)(head * p.group + (row - tok * (int32_t)p.group)) * p.q_head;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks) {
      const int d = (ks / S::kEB) * 32 * S::kEB + g * 8 * S::kEB + (ks % S::kEB) * 8;
      q[n][ks] = u32x4{0u, 0u, 0u, 0u};
      if (d < p.dim) q[n][ks] = *reinterpret_cast<const u32x4*>(src + 2 * d);
    }
  }

  f32x4 acc[kDt][kNr];
  float m[kNr], l[kNr];
#pragma unroll
  for (int n = 0; n < kNr; ++n) {
    m[n] = kNegInf;
    l[n] = 0.0f;
#pragma unroll
    for (int dt = 0; dt < kDt; ++dt) acc[dt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int32_t* table = p.table + (int64_t)t.seq * p.table_stride;
  const int32_t kk = lane & 31;
  // The page of this lane's key of a step (lanes l and l + 32 take key l): -2
  // where no row of the tile sees the key.
  auto page_id = [&](int32_t step) -> int32_t {
    const int32_t key = t.key_of(step) + kk;
    if (key >= t.end || (key < t.low && key >= p.sinks)) return -2;
    int32_t page, off;
    key_page(p, key, &page, &off);
    return table[page];
  };

  u32x4 kr[2][S::kLoadsK], vr[S::kLoadsV];
  uint32_t kb[2][kFmt == kFmtFp4 ? S::kLoadsK : 1], vb[kFmt == kFmtFp4 ? S::kLoadsV : 1];
  uint32_t ok = 0;     // the step's keys that are there
  bool met_bad = false;

  // Places the step's keys and issues their loads.
  auto load_step = [&](int32_t step, int32_t page) {
    const int32_t key = t.key_of(step) + kk;
    int32_t ignore, off;
    key_page(p, key, &ignore, &off);
    const bool there = page >= 0 && page < p.num_pages;
    met_bad = met_bad || (page != -2 && !there);
    const Side& side = lane < 32 ? p.k : p.v;
    const int64_t at = (int64_t)page * side.page + (int64_t)off * side.offset + (int64_t)head * side.head;
    my.at[lane >> 5][kk] = there ? at : -1;
    if constexpr (kFmt == kFmtFp4)
      my.scale_at[lane >> 5][kk] =
          (int64_t)page * side.s_page + (int64_t)off * side.s_offset + (int64_t)head * side.s_head;
    if constexpr (kFmt == kFmtE4M3 || kFmt == kFmtE5M2) {
      float sc = 1.0f;
      if (dyn && there)
        sc = *reinterpret_cast<const float*>(
            side.scales + (int64_t)page * side.s_page + (int64_t)off * side.s_offset +
            (p.scale_kind == KVATTN_TOKEN_HEAD ? (int64_t)head * side.s_head : 0));
      my.scale[lane >> 5][kk] = sc;
    }
    ok = (uint32_t)__ballot(there);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t a = my.at[0][h * 16 + c16];
#pragma unroll
      for (int i = 0; i < S::kLoadsK; ++i) {
        const int d = i * 32 * S::kEB + g * 8 * S::kEB;
        u32x4 x = u32x4{0u, 0u, 0u, 0u};
        uint32_t b = 127;
        if (a >= 0 && d < p.dim) {
          if constexpr (kFmt == kFmt16) {
            x = *reinterpret_cast<const u32x4*>(p.k.data + a + 2 * d);
          } else if constexpr (kFmt == kFmtFp4) {
            if constexpr (S::kEB == 4) {
              x = *reinterpret_cast<const u32x4*>(p.k.data + a + d / 2);
            } else {
              const u32x2 y = *reinterpret_cast<const u32x2*>(p.k.data + a + d / 2);
              x.x = y.x;
              x.y = y.y;
            }
            b = p.k.scales[my.scale_at[0][h * 16 + c16] + d / 32];
          } else {
            x = *reinterpret_cast<const u32x4*>(p.k.data + a + d);
          }
        }
        kr[h][i] = x;
        if constexpr (kFmt == kFmtFp4) kb[h][i] = b;
      }
    }
#pragma unroll
    for (int i = 0; i < S::kLoadsV; ++i) {
      const int row = i * S::kRowsV + lane / S::kLanesV;
      const int d = (lane % S::kLanesV) * S::kVE;
      const int64_t a = my.at[1][row];
      u32x4 x = u32x4{0u, 0u, 0u, 0u};
      uint32_t b = 127;
      if (a >= 0 && d < p.dim) {
        x = *reinterpret_cast<const u32x4*>(p.v.data + a + (kFmt == kFmt16 ? 2 * d : kFmt == kFmtFp4 ? d / 2 : d));
        if constexpr (kFmt == kFmtFp4) b = p.v.scales[my.scale_at[1][row] + d / 32];
      }
      vr[i] = x;
      if constexpr (kFmt == kFmtFp4) vb[i] = b;
    }
  };

  // V of the step into LDS as 16-bit values.
  auto store_v = [&]() {
#pragma unroll
    for (int i = 0; i < S::kLoadsV; ++i) {
      const int row = i * S::kRowsV + lane / S::kLanesV;
      uint8_t* dst = my.v + row * S::kStrideV + (lane % S::kLanesV) * S::kVE * 2;
      if constexpr (kFmt == kFmt16) {
        *reinterpret_cast<u32x4*>(dst) = vr[i];
      } else if constexpr (kFmt == kFmtFp4) {
        const float sc = __uint_as_float(vb[i] << 23);
        const uint32_t x[4] = {vr[i].x, vr[i].y, vr[i].z, vr[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<u32x4*>(dst + 16 * e) = values8<kFp16, kFmt>(x[e], 0, sc);
      } else {
        // The scale's power of two goes into the values, exactly; its
        // significand into the weights.
        const float sc = my.scale[1][row];
        *reinterpret_cast<u32x4*>(dst) = values8<kFp16, kFmt>(vr[i].x, vr[i].y, sc);
        *reinterpret_cast<u32x4*>(dst + 16) = values8<kFp16, kFmt>(vr[i].z, vr[i].w, sc);
      }
    }
  };

  int32_t step = s_begin + (int32_t)w;
  int32_t page_next = -2;
  if (step < s_end) {
    load_step(step, page_id(step));
    if (step + kWaves < s_end) page_next = page_id(step + kWaves);
  }
  for (; step < s_end; step += kWaves) {
    const int32_t key0 = t.key_of(step);
    const uint32_t ok_now = ok;
    store_v();

    // S^T, in 16-key halves.
    f32x4 s[2][kNr];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int n = 0; n < kNr; ++n) s[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
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
#pragma unroll
        for (int n = 0; n < kNr; ++n) s[h][n] = mfma16<kFp16>(a, q[n][ks], s[h][n]);
      }
    }

    // Scales of the lane's keys: 4g ... 4g + 3 of each half.
    f32x4 ksc[2], vsc[2];
    if constexpr (kFmt == kFmtE4M3 || kFmt == kFmtE5M2) {
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
      load_step(step + kWaves, page_next);
      if (step + 2 * kWaves < s_end) page_next = page_id(step + 2 * kWaves);
    }

    // Some row does not see some key of the step.
    const bool mixed = ok_now != 0xFFFFFFFFu || key0 + kStep - 1 > t.p_lo ||
                       !(t.p_hi - key0 < p.window || key0 + kStep - 1 < p.sinks);
    uint32_t seen[kNr];   // bit 4 h + i: the row sees the lane's key i of half h
    u32x4 pt[kNr];        // P^T operand
#pragma unroll
    for (int n = 0; n < kNr; ++n) {
      float x[8];
      float top = kNegInf;
      seen[n] = 0xFFu;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[4 * h + i] = s[h][n][i] * (dyn ? c * ksc[h][i] : c);
      if (mixed) {
        seen[n] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t j = (i >> 2) * 16 + 4 * g + (i & 3);
          const bool see = ((ok_now >> j) & 1u) && sees(p, pos[n], key0 + j);
          x[i] = see ? x[i] : kNegInf;
          seen[n] |= see ? 1u << i : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, x[i]);
      if (__ballot(top > m[n] + kLazy || (m[n] == kNegInf && top > kNegInf)) != 0) {
        const float was = m[n], now = fmaxf(was, group_max4(top));
        const float f = now == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(was - now);
        m[n] = now;
        l[n] *= f;
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[dt][n][i] *= f;
      }
      const float base = m[n] == kNegInf ? 0.0f : m[n];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __builtin_amdgcn_exp2f(x[i] - base);
        l[n] += x[i];
      }
      if (dyn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = x[i] * vsc[i >> 2][i & 3];
          x[i] = (seen[n] >> i) & 1u ? y : 0.0f;
        }
      }
      pt[n] = u32x4{pack_pair<kFp16>(x[0], x[1]), pack_pair<kFp16>(x[2], x[3]),
                    pack_pair<kFp16>(x[4], x[5]), pack_pair<kFp16>(x[6], x[7])};
    }

    // O^T += V^T P^T.
    __builtin_amdgcn_wave_barrier();
    uint8_t* const col = my.v + (4 * g + (c16 >> 2)) * S::kStrideV + (c16 & 3) * 8;
    u32x4 vt[kDt];
#pragma unroll
    for (int dt = 0; dt < kDt; ++dt) {
      const u32x2 a = read_column4(col + dt * 32);
      const u32x2 b = read_column4(col + 16 * S::kStrideV + dt * 32);
      vt[dt] = u32x4{a.x, a.y, b.x, b.y};
    }
    bool apart = false;
    if (mixed && t.p_lo != t.p_hi) {
      // Rows see different keys.  0 * V is not 0 where V holds a NaN or an
      // infinity, which must not reach the rows that do not see it.
      f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) z = mfma16<kFp16>(vt[dt], u32x4{0u, 0u, 0u, 0u}, z);
      const float zz = z[0] + z[1] + z[2] + z[3];
      apart = __ballot(!(zz == 0.0f)) != 0;
    }
    if (!apart) {
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
        for (int n = 0; n < kNr; ++n) acc[dt][n] = mfma16<kFp16>(vt[dt], pt[n], acc[dt][n]);
    } else {
      // One key at a time, added to the rows that see it.
      for (int j = 0; j < kStep; ++j) {
        const int h = j >> 4, gj = (j >> 2) & 3, e = 4 * h + (j & 3);
        const bool mine = (int)g == gj;
        // the pair of the operand that holds the key, and the half of the pair
        const uint32_t keep = mine ? ((e & 1) ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
#pragma unroll
        for (int n = 0; n < kNr; ++n) {
          const uint32_t in[4] = {pt[n].x, pt[n].y, pt[n].z, pt[n].w};
          u32x4 one = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int k = 0; k < 4; ++k) one[k] = (e >> 1) == k ? in[k] & keep : 0u;
          const bool see = ((ok_now >> j) & 1u) && sees(p, pos[n], key0 + j);
#pragma unroll
          for (int dt = 0; dt < kDt; ++dt) {
            u32x4 va = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int k = 0; k < 4; ++k) va[k] = (e >> 1) == k ? vt[dt][k] & keep : 0u;
            const f32x4 y = mfma16<kFp16>(va, one, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[dt][n][i] += see ? y[i] : 0.0f;
          }
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (__ballot(met_bad) != 0 && head == 0 && lane == 0)
    report(p.flag, (uint32_t)(t.token0 + t.row0 / (int32_t)p.group));

  // Join the waves.
#pragma unroll
  for (int n = 0; n < kNr; ++n) {
    l[n] += __shfl_xor(l[n], 16);
    l[n] += __shfl_xor(l[n], 32);
    if (g == 0) {
      s_m[w][n * 16 + c16] = m[n];
      s_l[w][n * 16 + c16] = l[n];
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kNr; ++n) {
    if (n > 0) __syncthreads();
    if (n * 16 >= t.rows) return;   // the whole block
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) top = fmaxf(top, s_m[i][n * 16 + c16]);
    const float f = m[n] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[n] - top);
    float* o = reinterpret_cast<float*>(my.v) + c16 * S::kStrideO + 4 * g;
#pragma unroll
    for (int dt = 0; dt < kDt; ++dt) {
      f32x4 y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = acc[dt][n][i] * f;
      *reinterpret_cast<f32x4*>(o + dt * 16) = y;
    }
    __syncthreads();
    // 16 threads per row, four columns at a time
    const int r = threadIdx.x >> 4, part = threadIdx.x & 15;
    if (n * 16 + r < t.rows) {
      float row_top = kNegInf, row_l = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) row_top = fmaxf(row_top, s_m[i][n * 16 + r]);
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        const float mi = s_m[i][n * 16 + r];
        row_l += mi == kNegInf ? 0.0f : s_l[i][n * 16 + r] * __builtin_amdgcn_exp2f(mi - row_top);
      }
      const Row x = row_of(p, t, head, n * 16 + r);
      const int64_t at = x.index * p.splits + blockIdx.y;
      const float inv = row_l == 0.0f ? 0.0f : v_scale / row_l;
#pragma unroll
      for (int d = part * 4; d < kDim; d += 64) {
        f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
          y += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds[i].v) +
                                               r * S::kStrideO + d);
        if (d >= p.dim) continue;
        if (n_splits == 1) {
          *reinterpret_cast<u32x2*>(p.out + x.token * p.o_token + (int64_t)x.head * p.o_head + 2 * d) =
              u32x2{pack_pair<kFp16>(y[0] * inv, y[1] * inv), pack_pair<kFp16>(y[2] * inv, y[3] * inv)};
        } else {
          *reinterpret_cast<f32x4*>(p.ws_o + at * p.dim + d) = y;
        }
      }
      if (n_splits > 1 && part == 0) {
        p.ws_ml[2 * at] = row_top;
        p.ws_ml[2 * at + 1] = row_l;
      }
    }
  }
}

template <int kNr>
__global__ __launch_bounds__(256) void kvattn_join_kernel(const Params p) {
  const bool tensor = (kFmt == kFmtE4M3 || kFmt == kFmtE5M2) && p.scale_kind == KVATTN_TENSOR;
  join_splits<kFp16, kStep>(p, 16 * kNr, tensor && p.v.scales
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

template <int kNr>
int launch_nr(const Params& p, int padded_dim, hipStream_t stream) {
  const dim3 grid(p.tile_slots * p.kv_heads, (uint32_t)p.splits);
  void (*kernel)(Params) = padded_dim == 64    ? kvattn_split_kernel<64, kNr>
                           : padded_dim == 128 ? kvattn_split_kernel<128, kNr>
                                               : kvattn_split_kernel<256, kNr>;
  const int st = run(kernel, grid, p, stream);
  if (st != KVSTORE_OK || p.splits == 1) return st;
  return run(kvattn_join_kernel<kNr>, dim3(p.tile_slots * p.kv_heads), p, stream);
}

}  // namespace

#define KVATTN_NAME2(src, fmt) launch_split_##src##_##fmt
#define KVATTN_NAME(src, fmt) KVATTN_NAME2(src, fmt)
#if KVATTN_FP16
#define KVATTN_SRC fp16
#else
#define KVATTN_SRC bf16
#endif

int KVATTN_NAME(KVATTN_SRC, KVATTN_FMT)(const Params& p, int padded_dim, int nr,
                                        hipStream_t stream) {
  switch (nr) {
    case 1: return launch_nr<1>(p, padded_dim, stream);
    case 2: return launch_nr<2>(p, padded_dim, stream);
    default: return launch_nr<4>(p, padded_dim, stream);
  }
}

}  // namespace kvattn
