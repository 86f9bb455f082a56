// Paged attention for many rows (prompts, chunks of them, short runs), and for few
// where a 16-bit cache has much to read: compiled once per source type and cache
// format (KVATTN_FP16, KVATTN_FMT).
//
//   out = sum_k softmax_k(c q . K_k) V_k over the keys that a row sees.
//
// A block owns 128 rows (tokens x q heads of one kv head, so that the heads of
// a group share the keys that the block reads) and walks their keys in steps of
// 64; each of its four waves has 32 rows.  K and V go through LDS as 16-bit
// values, double-buffered: the next step's rows are on their way during a step's
// products (16 bits: straight into LDS; others in registers, converted and
// written behind the products), with one barrier a step.  The addresses of a
// step's rows (page table lookups) are worked out three steps ahead, one key a
// thread, and handed over through LDS.
//
// S^T = K Q^T on 32x32x16 MFMAs; a lane then holds keys of one row only, so the
// softmax needs one exchange between two lanes, and its weights are in place
// as the operand P^T of O^T = V^T P^T once the keys of V are taken in the same
// order: four consecutive ones at a time, by transposing reads.
//
// The running maximum is raised only when a score exceeds it by more than 2^8, as
// in the split kernel.
//
// Bound, at 128 dims, by a step's serial parts: 32 MFMAs (1024 cycles a wave), 32
// exponentials at quarter rate and some 150 other vector operations, reads of 32
// KB of LDS for each wave, two waves a SIMD.  A prompt of 8192 bf16 tokens (32 q
// heads on 8 of 128 dims, 550 GFLOP) takes 610-630 us, 0.87-0.90 PFLOP/s, where a
// matrix product of 8192^3 reaches 1.25; without the softmax it takes 0.93 of
// that time, without LDS reads 0.85, without loads and lookups 0.83, without all
// three 0.55.  Chunks of 2048 tokens over 8192 4-bit keys (324 GFLOP) take 366
// us.  Six chunks of up to 1024 tokens in windows of 2048 e4m3fn keys with a scale
// for each token and head (64 dims, 22 GFLOP) take 84 us: 372 blocks of 35 steps,
// 5300 cycles each, of which the lookup of addresses and scales takes 900 in the
// two waves that do it (the others wait), the products of Q and K 1000, the
// softmax and the products with V 1800, the conversion of the next rows 900.
#include "attention_device.h"
#include "kvstore.h"

namespace kvattn {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr bool kFp16 = KVATTN_FP16 != 0;
constexpr int kFmt = KVATTN_FMT;
constexpr bool kFp8 = kFmt == kFmtE4M3 || kFmt == kFmtE5M2;
constexpr float kLazy = 8.0f;
constexpr int kStep = kTileStep;
constexpr int kRing = 4;   // steps whose row addresses are kept

// 16-bit rows of kDim dims are loaded straight into LDS (kDirect), with no
// registers in between.  Such loads fill LDS in the order of the lanes, so rows
// cannot be padded; instead the 16-byte pieces of a row change places with the
// row's number, which keeps the reads of neighbouring rows on different banks.
template <int kDim, bool kDirect>
struct Shape {
  static constexpr int kElems = kFmt == kFmt16 ? 8 : kFmt == kFmtFp4 ? 32 : 16;   // of 16 bytes
  static constexpr int kLanes = kDim / kElems;                 // threads per row
  static constexpr int kRows = kThreads / kLanes;              // rows per access of the block
  static constexpr int kLoads = kRows >= kStep ? 1 : kStep / kRows;
  static constexpr int kStrideK = 2 * kDim + (kDirect ? 0 : 16);   // bytes of a row in LDS
  static constexpr int kStrideV = 2 * kDim + (kDirect ? 0 : 32);
  static constexpr int kPieces = kDim / 8;                     // of 16 bytes, of a row
  // Place of a K row's piece, and of a V row's (whose pairs stay together: a
  // transposing read takes 32 bytes of each of four rows).
  static constexpr uint32_t place_k(uint32_t row) { return kDirect ? row & (kPieces < 16 ? kPieces - 1 : 15) : 0; }
  static constexpr uint32_t place_v(uint32_t row) { return kDirect ? 2 * (row & (kPieces < 16 ? 3 : 7)) : 0; }
};

template <int kDim, bool kDirect>
struct Lds {
  alignas(256) uint8_t k[2][kStep * Shape<kDim, kDirect>::kStrideK];
  alignas(256) uint8_t v[2][kStep * Shape<kDim, kDirect>::kStrideV];
  uint64_t at[kRing][2][kStep];        // addresses of K and V rows
  uint64_t scale_at[kFmt == kFmtFp4 ? kRing : 1][2][kFmt == kFmtFp4 ? kStep : 1];
  alignas(16) float scale[kFp8 ? kRing : 1][2][kFp8 ? kStep : 4];
  alignas(16) float v_sig[kFp8 ? kRing : 1][kFp8 ? kStep : 4];   // significands of V's
  unsigned long long ok[kRing];        // keys that are there
};

template <int kDim, bool kFull>
__global__ __launch_bounds__(kThreads, kDim <= 128 ? 2 : 1) void kvattn_tile_kernel(const Params p) {
  constexpr bool kDirect = kFull && kFmt == kFmt16;
  typedef Shape<kDim, kDirect> S;
  const int32_t dim = kFull ? kDim : p.dim;
  constexpr int kKs = kDim / 16;    // k steps of Q K^T
  constexpr int kDt = kDim / 32;    // column tiles of O
  __shared__ Lds<kDim, kDirect> lds;

  const uint32_t head = blockIdx.x % p.kv_heads;
  // later tiles of a sequence see more keys: they start first
  const uint32_t slot = p.tile_slots - 1 - blockIdx.x / p.kv_heads;
  const uint32_t tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const uint32_t half = lane >> 5, c32 = lane & 31, c16 = lane & 15;
  Tile<kStep> t;
  if (!tile_of(p, slot, kTileRows, &t)) return;
  int32_t n_splits;
  const int32_t chunk = split_steps(p, t, &n_splits);
  if ((int32_t)blockIdx.y >= n_splits) return;
  const int32_t s_begin = blockIdx.y * chunk;
  const int32_t s_end = min(t.steps, s_begin + chunk);

  const bool dyn = kFp8 && p.scale_kind != KVATTN_TENSOR;
  float c = p.scale2, v_scale = 1.0f;
  if (kFp8 && !dyn) {
    if (p.k.scales) c *= *reinterpret_cast<const float*>(p.k.scales);
    if (p.v.scales) v_scale = *reinterpret_cast<const float*>(p.v.scales);
  }
  // The softmax below wants c > 0: a negative one turns the signs of q (exactly),
  // and for 0 a tiny one does (all weights equal, masked scores still -inf).
  const uint32_t flip = c < 0.0f ? 0x80008000u : 0u;
  c = __builtin_fabsf(c);
  if (c == 0.0f) c = 1e-37f;

  // Q^T operand of this lane's row.
  const int32_t my_row = w * 32 + c32;
  u32x4 q[kKs];
  int32_t pos;
  {
    const int32_t row = t.row0 + (my_row < t.rows ? my_row : t.rows - 1);
    const int32_t tok = row / (int32_t)p.group;
    pos = t.first_pos + tok;
    const uint8_t* src = p.q + (int64_t)(t.token0 + tok) * p.q_token +
                         (int64_t)(head * p.group + (row - tok * (int32_t)p.group)) * p.q_head;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks) {
      const int d = ks * 16 + half * 8;
      q[ks] = u32x4{0u, 0u, 0u, 0u};
      if (d < dim) q[ks] = *reinterpret_cast<const u32x4*>(src + 2 * d);
      q[ks] ^= flip;
    }
  }

  f32x16 acc[kDt];
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[dt][i] = 0.0f;
  float m = kNegInf, l = 0.0f;   // of this lane's keys; m is the same in lanes l, l ^ 32

  // --- row addresses: threads 0-63 take a step's K rows, 64-127 its V rows ---
  const int32_t* table = p.table + (int64_t)t.seq * p.table_stride;
  const bool looks = w <= 1, is_v = w == 1;
  const uint64_t page_bytes = is_v ? p.v.page : p.k.page, row_bytes = is_v ? p.v.offset : p.k.offset;
  const uint64_t page_scales = is_v ? p.v.s_page : p.k.s_page;
  const uint64_t row_scales = is_v ? p.v.s_offset : p.k.s_offset;
  const uint64_t rows_at =
      reinterpret_cast<uint64_t>(is_v ? p.v.data : p.k.data) + (int64_t)head * (is_v ? p.v.head : p.k.head);
  const uint64_t scales_at =
      reinterpret_cast<uint64_t>(is_v ? p.v.scales : p.k.scales) +
      (kFmt == kFmtFp4 || p.scale_kind == KVATTN_TOKEN_HEAD ? (int64_t)head * (is_v ? p.v.s_head : p.k.s_head)
                                                            : 0);
  bool met_bad = false;
  // Both loads below are made whether the key is one of the tile's or not, from a
  // place that is there: loads under a condition would be waited for at once.
  auto page_id = [&](int32_t step) -> int32_t {
    const int32_t key = t.key_of(step) + (int32_t)lane;
    int32_t page, off;
    key_page(p, key < t.end ? key : t.end - 1, &page, &off);
    return load_global<int32_t>(reinterpret_cast<uint64_t>(table + page));
  };
  // A step's scales are loaded by place and written to LDS a step later.
  struct Scale {
    float value;
    bool there;
  };
  auto put_scales = [&](int32_t step, Scale x) {
    if constexpr (kFp8) {
      const int r = (step - s_begin) & (kRing - 1);
      const float scale = dyn && x.there ? x.value : 1.0f;
      lds.scale[r][w][lane] = scale;
      if (is_v)
        lds.v_sig[r][lane] = __uint_as_float((__float_as_uint(scale) & 0x807FFFFFu) | 0x3F800000u);
    }
  };
  auto place = [&](int32_t step, int32_t page) -> Scale {
    const int32_t key = t.key_of(step) + (int32_t)lane;
    int32_t ignore, off;
    key_page(p, key, &ignore, &off);
    const bool want = step < s_end && key < t.end && (key >= t.low || key < p.sinks);
    const bool there = want && (uint32_t)page < (uint32_t)p.num_pages;
    met_bad = met_bad || (want && !there);
    const int r = (step - s_begin) & (kRing - 1);
    // Slot 0 stands in for keys that are not there: its row is loaded and not used.
    const uint64_t pg = there ? (uint32_t)page : 0, of = there ? (uint32_t)off : 0;
    const uint64_t sc_at = scales_at + pg * page_scales + of * row_scales;
    lds.at[r][w][lane] = rows_at + pg * page_bytes + of * row_bytes;
    if constexpr (kFmt == kFmtFp4) lds.scale_at[r][w][lane] = sc_at;
    const unsigned long long ok = __ballot(there);
    if (tid == 0) lds.ok[r] = ok;
    Scale x = {1.0f, there};
    if (dyn) x.value = load_global<float>(sc_at);
    return x;
  };

  // --- rows: global memory -> registers -> LDS ---
  u32x4 kr[S::kLoads], vr[S::kLoads];
  uint32_t kb[S::kLoads], vb[S::kLoads];
  // Threads past the step's rows or the head's dims load a row's start and
  // write nothing.
  const int32_t row0 = tid / S::kLanes, col = (tid % S::kLanes) * S::kElems;
  const bool writes = col < dim && row0 < kStep;
  const uint32_t piece = tid % S::kLanes;
  const uint32_t from = writes ? (kFmt == kFmt16 ? 2 * col : kFmt == kFmtFp4 ? col / 2 : col) : 0;
  auto load_rows = [&](int32_t step) {
    const int b = (step - s_begin) & 1, r = (step - s_begin) & (kRing - 1);
    // all addresses first: reads of LDS wait for loads into it
    uint64_t k_at[S::kLoads], v_at[S::kLoads];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int row = (row0 & (kStep - 1)) + i * S::kRows;
      k_at[i] = lds.at[r][0][row] + (kDirect ? 16 * (piece ^ S::place_k(row)) : from);
      v_at[i] = lds.at[r][1][row] + (kDirect ? 16 * (piece ^ S::place_v(row)) : from);
    }
    if constexpr (kDirect) {
      // keeps the reads above from being moved down
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) asm volatile("" : "+v"(k_at[i]), "+v"(v_at[i]));
    }
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int row = (row0 & (kStep - 1)) + i * S::kRows;
      if constexpr (kDirect) {
        const int to = (i * S::kRows + w * (S::kRows / kWaves)) * S::kStrideK;   // of the wave
        load_to_lds(k_at[i], lds.k[b] + to);
        load_to_lds(v_at[i], lds.v[b] + to);
      } else {
        kr[i] = load_global<u32x4>(k_at[i]);
        vr[i] = load_global<u32x4>(v_at[i]);
        if constexpr (kFmt == kFmtFp4) {
          kb[i] = load_global<uint8_t>(lds.scale_at[r][0][row] + (writes ? col / 32 : 0));
          vb[i] = load_global<uint8_t>(lds.scale_at[r][1][row] + (writes ? col / 32 : 0));
        }
      }
    }
  };
  // Some row of the tile does not see some key of the step.
  auto mixed_step = [&](int32_t step, unsigned long long ok) {
    const int32_t key0 = t.key_of(step);
    return ok != ~0ull || key0 + kStep - 1 > t.p_lo ||
           !(t.p_hi - key0 < p.window || key0 + kStep - 1 < p.sinks);
  };
  // Where rows see different keys, NaN and infinities of V (0 * V is not 0 for
  // them) are left out of the product, and added at the end to the rows that do
  // see them.
  const bool ragged = t.p_lo != t.p_hi;
  bool special = false;
  auto put = [&](uint8_t* dst, u32x4 x, uint32_t byte, float sc, bool clean) {
    if constexpr (kFmt == kFmt16) {
      if (clean) x = finite8<kFp16>(x, &special);
      *reinterpret_cast<u32x4*>(dst) = x;
    } else if constexpr (kFmt == kFmtFp4) {
      if (clean && byte == 255) {
        special = true;
        byte = 127;
        x = u32x4{0u, 0u, 0u, 0u};
      }
      const float s4 = __uint_as_float(byte << 23);
      const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x4*>(dst + 16 * i) = values8<kFp16, kFmt>(e[i], 0, s4);
    } else {
      u32x4 a = values8<kFp16, kFmt>(x.x, x.y, sc), b = values8<kFp16, kFmt>(x.z, x.w, sc);
      if (clean) {
        a = finite8<kFp16>(a, &special);
        b = finite8<kFp16>(b, &special);
      }
      *reinterpret_cast<u32x4*>(dst) = a;
      *reinterpret_cast<u32x4*>(dst + 16) = b;
    }
  };
  auto store_rows = [&](int32_t step) {
    const int b = (step - s_begin) & 1, r = (step - s_begin) & (kRing - 1);
    const unsigned long long ok = lds.ok[r];
    const bool clean = ragged && mixed_step(step, ok);
    if constexpr (kDirect) {
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's rows are in LDS
      if (ok == ~0ull && !clean) return;
      // each lane puts right what it loaded
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        const int row = row0 + i * S::kRows;
        u32x4* at = reinterpret_cast<u32x4*>(lds.v[b] + row * S::kStrideV + 16 * piece);
        u32x4 x = *at;
        if (clean) x = finite8<kFp16>(x, &special);
        *at = (ok >> row) & 1ull ? x : u32x4{0u, 0u, 0u, 0u};
      }
      return;
    }
    if (ok != ~0ull) {   // 0 * V must be 0 for keys that are not there
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        const bool there = (ok >> (row0 + i * S::kRows)) & 1ull;
        vr[i] = there ? vr[i] : u32x4{0u, 0u, 0u, 0u};
        if constexpr (kFmt == kFmtFp4) vb[i] = there ? vb[i] : 127u;
      }
    }
    if (!writes) return;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int row = row0 + i * S::kRows;
      put(lds.k[b] + row * S::kStrideK + 2 * col, kr[i], kb[i], 1.0f, false);
      // V's power of two goes into the values, exactly; its significand into the weights
      put(lds.v[b] + row * S::kStrideV + 2 * col, vr[i], vb[i],
          kFp8 ? lds.scale[kFp8 ? r : 0][1][kFp8 ? row : 0] : 1.0f, clean);
    }
  };

  if (!kFull) {   // the columns that no thread writes
    u32x4* const all = reinterpret_cast<u32x4*>(lds.k[0]);
    for (uint32_t i = tid; i < (sizeof(lds.k) + sizeof(lds.v)) / 16; i += kThreads)
      all[i] = u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  int32_t page_next = 0;
  Scale scale_next = {1.0f, false};
  if (s_begin < s_end && looks) {
    const int32_t id0 = page_id(s_begin), id1 = page_id(s_begin + 1), id2 = page_id(s_begin + 2);
    page_next = page_id(s_begin + 3);
    const Scale x = place(s_begin, id0), y = place(s_begin + 1, id1);
    scale_next = place(s_begin + 2, id2);
    put_scales(s_begin, x);
    put_scales(s_begin + 1, y);
  }
  __syncthreads();
  if (s_begin < s_end) {
    load_rows(s_begin);
    store_rows(s_begin);
  }
  __syncthreads();

  for (int32_t step = s_begin; step < s_end; ++step) {
    const int b = (step - s_begin) & 1, r = (step - s_begin) & (kRing - 1);
    const int32_t key0 = t.key_of(step);
    const bool more = step + 1 < s_end;
    // What this waits for was loaded a step ago; after load_rows it would wait for
    // its loads, too.
    if (looks) {
      put_scales(step + 2, scale_next);
      scale_next = place(step + 3, page_next);
      page_next = page_id(step + 4);
    }
    if (more) load_rows(step + 1);

    // The step in 32-key halves, so that matrix and vector work of different
    // halves overlap within the wave: while the second half's products run, the
    // first's weights are worked out, and the other way round for V.
    const unsigned long long ok = lds.ok[r];
    const bool mixed = mixed_step(step, ok);
    // Rows 32 h + c32 of K; rows 16 k + 8 u + v_row of V (whose places are those
    // of rows c32 and v_row).
    const uint32_t v_row = 4 * half + (c16 >> 2);
    const uint8_t* const kp = lds.k[b] + c32 * S::kStrideK;
    uint8_t* const vp = lds.v[b] + v_row * S::kStrideV + 8 * (c16 & 1);
    auto k_operand = [&](int h, int ks) {
      const uint32_t at = 16 * ((2 * ks + half) ^ S::place_k(c32));
      return *reinterpret_cast<const u32x4*>(kp + h * 32 * S::kStrideK + at);
    };
    auto v_operand = [&](int k, int dt) {
      const uint32_t at = 16 * ((4 * dt + 2 * ((lane >> 4) & 1) + ((c16 >> 1) & 1)) ^ S::place_v(v_row));
      const u32x2 x = read_column4(vp + (16 * k) * S::kStrideV + at);
      const u32x2 y = read_column4(vp + (16 * k + 8) * S::kStrideV + at);
      return u32x4{x.x, x.y, y.x, y.y};
    };
    u32x4 pt[4];          // P^T operands of 16 keys each
    // Value i of half h: key key0 + 32 h + 8 (i / 4) + 4 half + i % 4.
    f32x16 s[2];
    uint32_t seen[2] = {~0u, ~0u};   // bit 8 (i / 4) + i % 4 of half h: the row sees value i
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[h][i] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] = mfma32<kFp16>(k_operand(h, ks), q[ks], s[h]);
    if constexpr (kFp8) {
      if (dyn) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 ks = *reinterpret_cast<const f32x4*>(&lds.scale[r][0][32 * h + 8 * j + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[h][4 * j + i] *= ks[i];
          }
      }
    }
    if (mixed) {
      const unsigned long long bits = seen_bits(p, pos, key0, ok) >> (4 * half);
      seen[0] = (uint32_t)bits;
      seen[1] = (uint32_t)(bits >> 32);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[h][i] = seen[h] & (1u << (8 * (i >> 2) + (i & 3))) ? s[h][i] : kNegInf;
    }
    float top = kNegInf;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[h][i]);
    top *= c;
    if (__ballot(top > m + kLazy || (m == kNegInf && top > kNegInf)) != 0) {
      const float now = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
      const float f = now == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[dt][i] *= f;
    }
    // Scores -> weights, two P^T operands.
    auto weights_of = [&](int h, f32x16& s, uint32_t see) {
      const float base = m == kNegInf ? 0.0f : -m;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, base));
        l += s[i];
      }
      if constexpr (kFp8) {
        if (dyn) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 vs = *reinterpret_cast<const f32x4*>(&lds.v_sig[r][32 * h + 8 * j + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * j + i] *= vs[i];
          }
          if (mixed) {    // the scale of a key that the row does not see may be anything
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = see & (1u << (8 * (i >> 2) + (i & 3))) ? s[i] : 0.0f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        pt[2 * h + k] = u32x4{pack_pair<kFp16>(s[8 * k], s[8 * k + 1]), pack_pair<kFp16>(s[8 * k + 2], s[8 * k + 3]),
                              pack_pair<kFp16>(s[8 * k + 4], s[8 * k + 5]), pack_pair<kFp16>(s[8 * k + 6], s[8 * k + 7])};
    };

    weights_of(0, s[0], seen[0]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) acc[dt] = mfma32<kFp16>(v_operand(k, dt), pt[k], acc[dt]);
    weights_of(1, s[1], seen[1]);
#pragma unroll
    for (int k = 2; k < 4; ++k)
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) acc[dt] = mfma32<kFp16>(v_operand(k, dt), pt[k], acc[dt]);

    if (more) store_rows(step + 1);
    __syncthreads();
  }
  if (__ballot(met_bad) != 0 && tid == 0 && head == 0)
    report(p.flag, (uint32_t)(t.token0 + t.row0 / (int32_t)p.group));

  if (__syncthreads_or(special)) {
    // Rare: V's NaN and infinities of the steps that they were left out of, for
    // the rows that see them.
    for (int32_t step = s_begin; step < s_end; ++step) {
      const int32_t key0 = t.key_of(step);
      for (int32_t key = key0; key < min(key0 + kStep, t.end); ++key) {
        if (key < t.low && key >= p.sinks) continue;
        int32_t page, off;
        key_page(p, key, &page, &off);
        page = table[page];
        if (page < 0 || page >= p.num_pages || !sees(p, pos, key)) continue;
        int32_t d0 = 4 * half;
        asm volatile("" : "+v"(d0));   // keeps 16 kDt comparisons from being carried along
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int32_t d = d0 + dt * 32 + 8 * (i >> 2) + (i & 3);
            if (d < dim) acc[dt][i] += special_at<kFmt, kFp16>(p, head, page, off, d);
          }
      }
    }
  }

  l += __shfl_xor(l, 32);
  if (my_row >= t.rows) return;
  const Row x = row_of(p, t, head, my_row);
  const int64_t at = x.index * p.splits + blockIdx.y;
  const float inv = l == 0.0f ? 0.0f : v_scale / l;
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = dt * 32 + 8 * j + 4 * half;
      if (d >= dim) continue;
      const f32x4 y = f32x4{acc[dt][4 * j], acc[dt][4 * j + 1], acc[dt][4 * j + 2], acc[dt][4 * j + 3]};
      if (n_splits == 1)
        *reinterpret_cast<u32x2*>(p.out + x.token * p.o_token + (int64_t)x.head * p.o_head + 2 * d) =
            u32x2{pack_pair<kFp16>(y[0] * inv, y[1] * inv), pack_pair<kFp16>(y[2] * inv, y[3] * inv)};
      else
        *reinterpret_cast<f32x4*>(p.ws_o + at * dim + d) = y;
    }
  if (n_splits > 1 && half == 0) {
    p.ws_ml[2 * at] = m;
    p.ws_ml[2 * at + 1] = l;
  }
}

__global__ __launch_bounds__(256) void kvattn_join_tiles_kernel(const Params p) {
  join_splits<kFp16, kStep>(p, kTileRows, kFp8 && p.scale_kind == KVATTN_TENSOR && p.v.scales
                                              ? *reinterpret_cast<const float*>(p.v.scales)
                                              : 1.0f);
}

int run(void (*kernel)(Params), dim3 grid, const Params& p, hipStream_t stream) {
  Params copy = p;
  void* argv[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(kThreads), argv, 0,
                         stream) == hipSuccess
             ? KVSTORE_OK
             : KVSTORE_ERR_HIP;
}

}  // namespace

#define KVATTN_NAME2(src, fmt) launch_tile_##src##_##fmt
#define KVATTN_NAME(src, fmt) KVATTN_NAME2(src, fmt)
#if KVATTN_FP16
#define KVATTN_SRC fp16
#else
#define KVATTN_SRC bf16
#endif

int KVATTN_NAME(KVATTN_SRC, KVATTN_FMT)(const Params& p, int padded_dim, hipStream_t stream) {
  const dim3 grid(p.tile_slots * p.kv_heads, (uint32_t)p.splits);
  const bool full = p.dim == padded_dim;
  void (*kernel)(Params) =
      padded_dim == 64    ? (full ? kvattn_tile_kernel<64, true> : kvattn_tile_kernel<64, false>)
      : padded_dim == 128 ? (full ? kvattn_tile_kernel<128, true> : kvattn_tile_kernel<128, false>)
                          : (full ? kvattn_tile_kernel<256, true> : kvattn_tile_kernel<256, false>);
  const int st = run(kernel, grid, p, stream);
  if (st != KVSTORE_OK || p.splits == 1) return st;
  return run(kvattn_join_tiles_kernel, dim3(p.tile_slots * p.kv_heads * p.join_parts), p,
             stream);
}

}  // namespace kvattn
