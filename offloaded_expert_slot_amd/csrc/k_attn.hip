// Attention of new tokens over a paged cache, and the weights that its entries receive.
//
// One pass over the cache with the running maximum and sum of the softmax.  A workgroup
// takes a tile of rows - (token, query head) pairs of one sequence and one cache head, so
// that every key and value read serves all query heads of its group - and goes over the
// entries that any of them sees.  Both products run on the matrix units, transposed:
//
//   S^T = K Q^T   (entries x rows)   A = keys from LDS, B = queries in registers
//   O^T = V^T P^T (dims x rows)      A = values from LDS, read transposed, B = weights
//
// In the accumulator of v_mfma_f32_32x32x16_bf16 a lane holds one column, so one row of
// the attention: its statistics are lane scalars, and the weights are in the lane that
// needs them as the next product's B operand, with no trip through LDS.  (Accumulator
// register i of lane (c, h) is entry 8 (i / 4) + 4 h + i % 4; the sum over entries may
// run in any order, so the V operand is read in that order.)
//
// Bound by the matrix units with many rows (2048 tokens x 32 heads over 24111 entries of 128 values: 0.80 ms, 970
// TFLOP/s; 0.76 ms a call), by reading the cache once in decode steps (32 sequences of 1 .. 16384 e4m3 entries: 30 us, 3.9 TB/s).  With
// a window of 128 (2023 tokens x 64 heads of 64 values) a tile sees some four tiles of entries, nearly all masked in
// part: 24 us, of them some 11 in each of two rounds of workgroups.
//
// Two shapes:
//   TILE    128 rows, 32 to each of 4 waves, which share tiles of 64 entries.  With few tiles
//           of rows the entries are split over several workgroups.
//   SPLIT   up to 32 rows (decode steps, small chunks), the same for all waves, each of
//           which goes over entries of its own, 32 at a time, with no barrier; the waves'
//           sums are joined through LDS.  The entries of all (tile, head) pairs, in units of
//           32 per wave, are cut into equal shares for as many workgroups as the GPU holds at
//           once, whatever the sequences' lengths (a grid over (tile, head, split) took 62 us
//           for 32 sequences of 1 .. 16384 entries, most of it short and empty workgroups).
// The sums of a pair that several workgroups share go through the workspace, and
// attn_merge_kernel joins them in order.
//
// Rows of LDS tiles are DP values (head_dim padded to 64, 128 or 256) in 16-byte chunks,
// chunk c of row r at c ^ swizzle(r), so that neither the 16-byte key reads (16 rows, one
// chunk) nor the transposing value reads (4 rows, 4 chunks) meet in a bank.  A bf16 cache
// goes to LDS with direct loads (each lane's global address carries page and swizzle);
// e4m3 goes through registers, where it becomes bf16 (exactly).  Entries that no row
// sees, bad pages and values behind head_dim are staged from a zero chunk.
//
// Weights are rounded to bf16 (the matrix product's type) with the row sum taken before
// the rounding.  Half a step (2^-8) of each weight is about what the rounding of the output
// to bf16 costs once more: 2048 tokens over 24111 entries lie 0.0024 from the 64-bit values
// (relative, in the root mean square), where fp32 weights leave the output's 0.0017.  Two
// bf16 parts a weight would take that away, at half as much matrix work again.

#include <algorithm>
#include <type_traits>

#include "layer_device.h"
#include "oes_internal.h"

namespace oes {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.f;   // a running maximum may be this much (log2) too small

__device__ __attribute__((aligned(16))) const uint32_t zero_chunk[4] = {0, 0, 0, 0};

template <int DP>
__device__ inline int swizzle(int row) {
  // DP = 64: two rows share the 256 bytes of all banks
  return DP == 64 ? ((row >> 1) & 1) << 2 | ((row >> 2) & 3) : (row & 3) << 2 | ((row >> 2) & 3);
}

// 16 bytes per lane from global memory to LDS base + 16 * lane; counted by vmcnt only
__device__ inline void load_to_lds(const void *src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory");
}
// the same with a wave-uniform base and a 32-bit offset per lane
__device__ inline void load_to_lds(const void *base, uint32_t off, uint32_t lds) {
  const uint64_t b = (uint64_t)base;
  const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)b);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(u) : "memory");
}
template <int N>
__device__ inline void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ inline uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}
// the value of the lane's other half (lane ^ 32) joined with its own
__device__ inline float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <bool HI>
__device__ inline uint32_t fp8_bf16_pair(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// Masks: bit e of 32 for the entries [lo, hi) of a row; and all bits of an accumulator register's entry (see the top).
// Bit to sign to select is two operations a score, where comparing took five.
__device__ inline uint32_t seen_bits(int lo, int hi) {
  return (uint32_t)((1ull << min(max(hi, 0), 32)) - 1) & ~(uint32_t)((1ull << min(max(lo, 0), 32)) - 1);
}
__device__ inline int seen_sign(uint32_t seen, int i) { return (int)(seen << (31 - (8 * (i / 4) + i % 4))) >> 31; }

// What a launch is cut into.
struct Plan {
  int tile_tokens;   // tokens of a tile
  int tiles;         // tiles of all sequences, at most
  int splits;        // TILE: parts of the entries, at most
  int chunk;         // TILE: entries of a part; SPLIT: entries of a unit, 1 << chunk_log
  int chunk_log;     // TILE: -1
  int blocks;        // SPLIT: workgroups
};

// A tile of rows and the entries that it sees.
struct Tile {
  int b, first, t0, tokens;    // sequence, its first row, the tile's first token and tokens
  int len, rows;               // entries and rows of the sequence
  int lo, hi;                  // entries that any row sees
  int lo_last, hi_first;       // entries that every row sees
  int base, parts;             // first entry of part (unit) 0; parts (units) that hold entries, at least 1
};

__device__ inline void tile_entries(const AttnArgs &a, const Plan &p, Tile &t) {
  t.tokens = min(p.tile_tokens, t.rows - t.t0);
  kv_seen(t.len, t.rows, t.t0, a.window, &t.lo, &t.hi_first);
  kv_seen(t.len, t.rows, t.t0 + t.tokens - 1, a.window, &t.lo_last, &t.hi);
  t.base = t.lo & ~31;
  const int span = t.hi - t.base + p.chunk - 1;
  t.parts = t.hi > t.base ? (p.chunk_log >= 0 ? span >> p.chunk_log : span / p.chunk) : 1;
}

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// Inclusive sum over the lanes up to this one: within rows of 16, then across them.
__device__ inline int scan64(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 to row 1, lane 47 to row 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
  return v;
}
__device__ inline int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// The lane's sequence b0 + lane: rows, entries; 0 where there is none.
__device__ inline void lane_sequence(const AttnArgs &a, int b0, int *first, int *rows, int *len) {
  const int b = b0 + (threadIdx.x & 63);
  *first = *rows = *len = 0;
  bool bad = false;
  if (b < a.kv.batch) {
    *rows = kv_rows(a.q_start[b], a.q_start[b + 1], a.n, first, &bad);
    *len = kv_len(a.kv, a.kv.len[b], &bad);
    if (bad) raise_status(a.kv);
  }
}
__device__ inline void take_sequence(Tile &t, int b0, int w, int first, int rows, int len) {
  t.b = b0 + w;
  t.first = lane_value(first, w);
  t.rows = lane_value(rows, w);
  t.len = lane_value(len, w);
}

// Tile `idx` in the order of the sequences (wave-wide; the same answer in every lane).
__device__ inline bool find_tile(const AttnArgs &a, const Plan &p, int idx, Tile &t) {
  int before = 0;
  for (int b0 = 0; b0 < a.kv.batch; b0 += 64) {
    int first, rows, len;
    lane_sequence(a, b0, &first, &rows, &len);
    const int mine = (rows + p.tile_tokens - 1) / p.tile_tokens, upto = before + scan64(mine);
    const uint64_t hit = __ballot(upto > idx && upto - mine <= idx);
    if (hit) {
      const int w = uniform(__builtin_ctzll(hit));
      take_sequence(t, b0, w, first, rows, len);
      t.t0 = (idx - lane_value(upto - mine, w)) * p.tile_tokens;
      tile_entries(a, p, t);
      return true;
    }
    before = lane_value(upto, 63);
  }
  return false;
}

// A (tile, head) pair costs a workgroup about as much as kBegin units before its first one (rows, pages, a
// latency each, and the joining of the waves), so it counts as kBegin + parts units, the first kBegin without
// entries.
constexpr int kBegin = 4;

// Units of a sequence, over its tiles and all cache heads.
__device__ inline int sequence_units(const AttnArgs &a, const Plan &p, int rows, int len) {
  int sum = 0;
  Tile t;
  t.rows = rows;
  t.len = len;
  for (t.t0 = 0; t.t0 < rows; t.t0 += p.tile_tokens) {
    tile_entries(a, p, t);
    sum += kBegin + t.parts;
  }
  return sum * a.kv.kv_heads;
}

// SPLIT's order of units: sequence, tile, head, entries.  The lane's sequence of the first 64, kept over the calls.
struct Scan {
  int first, rows, len, mine, upto;
};
__device__ inline Scan scan_sequences(const AttnArgs &a, const Plan &p, int b0, int before) {
  Scan s;
  lane_sequence(a, b0, &s.first, &s.rows, &s.len);
  s.mine = sequence_units(a, p, s.rows, s.len);
  s.upto = before + scan64(s.mine);
  return s;
}
__device__ inline int all_units(const AttnArgs &a, const Plan &p, const Scan &s0) {
  int total = lane_value(s0.upto, 63);
  for (int b0 = 64; b0 < a.kv.batch; b0 += 64) total = lane_value(scan_sequences(a, p, b0, total).upto, 63);
  return total;
}
// Where unit `u` stands: its tile, head and place `x` among the pair's units.  Wave-wide.  (There is one, unless ranges of
// rows that overlap have made the number of units wrap.)
__device__ inline bool find_unit(const AttnArgs &a, const Plan &p, const Scan &s0, int u, Tile &t, int *g, int *x) {
  Scan s = s0;
  for (int b0 = 0; b0 < a.kv.batch; b0 += 64) {
    if (b0) s = scan_sequences(a, p, b0, lane_value(s.upto, 63));
    const uint64_t hit = __ballot(s.upto > u && s.upto - s.mine <= u);
    if (!hit) continue;
    const int w = uniform(__builtin_ctzll(hit));
    take_sequence(t, b0, w, s.first, s.rows, s.len);
    int left = u - lane_value(s.upto - s.mine, w);
    for (t.t0 = 0;; t.t0 += p.tile_tokens) {
      tile_entries(a, p, t);
      const int all = (kBegin + t.parts) * a.kv.kv_heads;
      if (left < all) break;
      left -= all;
    }
    *g = left / (kBegin + t.parts);
    *x = left - *g * (kBegin + t.parts);
    return true;
  }
  return false;
}
// units of a workgroup
__device__ inline int unit_share(const Plan &p, int total) { return (total + p.blocks - 1) / p.blocks; }

// Partial sums.  TILE: ws holds [splits][n][q_heads] pairs (maximum in log2, sum), then as many rows of head_dim
// values.  SPLIT: the same of [blocks][2][32]: rows of the pair that a workgroup's share begins within (0), and of
// the one that its share ends within (1).
template <bool TILE>
__device__ inline float2 *part_stats(const AttnArgs &a, int64_t at) {
  return reinterpret_cast<float2 *>(a.ws) + at;
}
template <bool TILE>
__device__ inline float *part_sums(const AttnArgs &a, const Plan &p, int64_t at) {
  const int64_t rows = TILE ? (int64_t)p.splits * a.n * a.q_heads : (int64_t)p.blocks * 64;
  return a.ws + 2 * rows + at * a.kv.head_dim;
}

template <int DP, bool FP8, bool TILE>
struct Shape {
  static constexpr int waves = TILE ? 4 : (DP == 256 ? 2 : 4);
  static constexpr int entries = TILE ? 64 : 32;            // of an LDS tile
  // (64-wide heads: loads two tiles ahead, since a tile's products take less than a load)
  static constexpr int buffers = FP8 && !TILE ? 1 : (TILE && !FP8 && DP == 64 ? 3 : 2);
  static constexpr int copies = TILE ? 1 : waves;           // SPLIT: a tile per wave
  static constexpr int tile_bytes = entries * DP * 2;       // K; V as much again
  static constexpr int lds = copies * buffers * 2 * tile_bytes;
  static constexpr int own = TILE ? entries / waves : entries;  // rows that a wave stages
  // waves of a SIMD that registers and LDS are held to
  static constexpr int resident = DP == 256 ? 1 : (TILE || FP8 || DP == 64 ? 2 : 1);
};

template <int DP, bool FP8, bool TILE>
__global__ __launch_bounds__((Shape<DP, FP8, TILE>::waves * 64), (Shape<DP, FP8, TILE>::resident)) void attn_kernel(AttnArgs a, Plan plan) {
  using S = Shape<DP, FP8, TILE>;
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  constexpr int KT = S::entries / 32, NB = S::buffers, KS = DP / 16, DT = DP / 32, E = S::entries, es = FP8 ? 1 : 2;
  constexpr uint64_t kAll = E == 64 ? ~0ull : 0xffffffffull;
  __shared__ __attribute__((aligned(16))) uint8_t sm[S::lds];
  __shared__ float jm[4][32], jl[4][32];
  __shared__ int odd_sm, j_row[32], j_head[32];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 31, half = lane >> 5;
  const int D = a.kv.head_dim, G = a.q_heads / a.kv.kv_heads, shift = a.shift;
  const float cs = a.scale * a.kv.k_scale * kLog2e;

  // ---- lane constants of the staging
  constexpr int CPR = FP8 ? DP / 16 : DP / 8;   // chunks of a head row
  constexpr int RPI = 64 / CPR;                 // rows that a wave's load covers
  constexpr int LD = S::own / RPI;              // loads of a wave for k, and for v
  constexpr int own0 = TILE ? S::own : 0;       // rows of a tile before those that wave 1 stages
  constexpr int GR = S::own / 16, LG = 16 / RPI, NG = E / 16;   // groups of 16 rows; loads of a group
  uint8_t *tiles = sm + (TILE ? 0 : wave * NB * 2 * S::tile_bytes);
  // Whole tiles of pages of 16 entries and more: 16 rows stand in one page, so their addresses are a scalar base
  // and an offset that the lane keeps (with an address of its own per lane and load, 2048 tokens at 24111 entries took
  // 1.29 ms).  Page numbers are read a tile ahead, through the scalar cache.
  const bool paged16 = shift >= 4 && D == DP && (a.kv.k_row | a.kv.v_row) < (1 << 22);
  // (FP8: neighbouring lanes take different rows, whose bf16 chunks go to different banks)
  auto lane_row = [](int ln) { return FP8 ? ln % RPI : ln / CPR; };
  uint32_t k_lane[LG], v_lane[LG];
#pragma unroll
  for (int i = 0; i < LG; ++i) {
    const int row = i * RPI + lane_row(lane), ch = FP8 ? lane / RPI : (lane % CPR) ^ swizzle<DP>(row);
    k_lane[i] = (uint32_t)(row * a.kv.k_row) * es + ch * 16;
    v_lane[i] = (uint32_t)(row * a.kv.v_row) * es + ch * 16;
  }

  // ---- what this workgroup goes over: one part of a pair (TILE), or its share of the units (SPLIT)
  Tile t;
  Scan scan = {};
  int g = 0, split = 0, unit = 0, unit_end = 0;
  if (TILE) {
    // heads are the fastest index: neighbouring workgroups, on different XCDs, take different heads, so that an
    // XCD keeps to few of them; later tiles, which see more, come first
    int id = blockIdx.x;
    g = id % a.kv.kv_heads;
    id /= a.kv.kv_heads;
    split = id / plan.tiles;
    if (!find_tile(a, plan, plan.tiles - 1 - (id - split * plan.tiles), t) || split >= t.parts) return;
    if (threadIdx.x == 0) odd_sm = 0;
  } else {
    scan = scan_sequences(a, plan, 0, 0);
    const int total = all_units(a, plan, scan), share = unit_share(plan, total);
    unit = min((int64_t)blockIdx.x * share, (int64_t)total);
    unit_end = min((int64_t)unit + share, (int64_t)total);
    if (unit >= unit_end) return;
    g = a.kv.kv_heads;
  }
  do {
    int from, to, x = 0;
    bool direct;
    if (TILE) {
      from = t.base + split * plan.chunk;
      to = min(t.hi, from + plan.chunk);
      direct = t.parts == 1;
    } else {
      if (++g < a.kv.kv_heads)
        x = 0;   // the same tile's next head
      else if (!find_unit(a, plan, scan, unit, t, &g, &x))
        return;
      const int n = min(kBegin + t.parts - x, unit_end - unit), x1 = x + n - kBegin;
      unit += n;
      if (x1 <= 0) break;   // the share ends before the pair's first entries
      x = max(0, x - kBegin);
      from = t.base + x * plan.chunk;
      to = min(t.hi, t.base + x1 * plan.chunk);
      direct = x == 0 && x1 == t.parts;
    }
    const int32_t *table = a.kv.table + t.b * a.kv.table_stride;
    typedef __attribute__((address_space(4))) const int32_t const_i32;
    const const_i32 *ctable = (const const_i32 *)(uintptr_t)table;
    const uint8_t *kb = static_cast<const uint8_t *>(a.kv.k) + a.kv.k_head * g * es;
    const uint8_t *vb = static_cast<const uint8_t *>(a.kv.v) + a.kv.v_head * g * es;
    const int step = TILE ? E : E * S::waves, j_first = from + (TILE ? 0 : wave * E);

    // ---- this lane's row
    const int r = (TILE ? wave * 32 : 0) + c;
    const bool row_live = r < t.tokens * G;
    const int tok = r / G, row_t = t.first + t.t0 + tok, row_h = g * G + (r - tok * G);
    int lo = 0, hi = 0;
    if (row_live) kv_seen(t.len, t.rows, t.t0 + tok, a.window, &lo, &hi);
    bf16x8 q[KS];
    {
      const uint16_t *qp = a.q.p + row_t * a.q.row + row_h * a.q.head + 8 * half;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        u32x4 v = {0, 0, 0, 0};
        if (row_live && ks * 16 < D) v = *reinterpret_cast<const u32x4 *>(qp + 16 * ks);
        q[ks] = __builtin_bit_cast(bf16x8, v);
      }
    }
    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    float m = -INFINITY, l = 0.f;

    // ---- staging
    u32x4 stage_k[FP8 ? LD : 1], stage_v[FP8 ? LD : 1];
    int pages[NG];
    auto peek = [&](int j0) {  // pages of the tile at j0, where the tile is whole
      if (paged16 && j0 >= t.lo && j0 + E <= to) {
#pragma unroll
        for (int y = 0; y < NG; ++y) pages[y] = ctable[(j0 + 16 * y) >> shift];
      }
    };
    // Loads of the tile at j0 into buffer `buf`; returns which of its entries there are.
    auto issue = [&](int j0, int buf) -> uint64_t {
      uint8_t *dst = tiles + buf * 2 * S::tile_bytes + wave * own0 * DP * 2;
      if (paged16 && j0 >= t.lo && j0 + E <= to) {
        bool ok = true;
#pragma unroll
        for (int y = 0; y < NG; ++y) ok &= (uint32_t)pages[y] < (uint32_t)a.kv.num_pages;
        if (ok) {
#pragma unroll
          for (int z = 0; z < GR; ++z) {
            int page = pages[z];
            if (TILE) {
#pragma unroll
              for (int y = 1; y < NG; ++y)
                if (wave == y) page = pages[y];
            }
            const int in_page = (j0 + wave * own0 + 16 * z) & (a.kv.page_size - 1);
            const uint8_t *kp = kb + kv_k_off(a.kv, page, in_page) * es, *vp = vb + kv_v_off(a.kv, page, in_page) * es;
#pragma unroll
            for (int i = 0; i < LG; ++i) {
              if (FP8) {
                stage_k[z * LG + i] = *reinterpret_cast<const u32x4 *>(kp + k_lane[i]);
                stage_v[z * LG + i] = *reinterpret_cast<const u32x4 *>(vp + v_lane[i]);
              } else {
                const uint32_t at = uniform(lds_addr(dst + (16 * z + i * RPI) * DP * 2));
                load_to_lds(kp, k_lane[i], at);
                load_to_lds(vp, v_lane[i], at + S::tile_bytes);
              }
            }
          }
          return ~0ull;
        }
      }
      // one entry per lane, zeros where there is none.  (The lane is made opaque: what this rare path computes
      // from it is not to live in registers through the loop.)
      int ln = lane;
      asm volatile("" : "+v"(ln));
      const int j = j0 + (E == 32 ? ln & 31 : ln);
      int page = -1, in_page = 0;
      if (j >= t.lo && j < to) {
        page = kv_page(a.kv, table, shift, j, &in_page);
        if (page < 0) raise_status(a.kv);
      }
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int row = wave * own0 + i * RPI + lane_row(ln), ch = FP8 ? ln / RPI : (ln % CPR) ^ swizzle<DP>(row);
        const int pg = __shfl(page, row, 64), ip = __shfl(in_page, row, 64);
        const uint8_t *ks = reinterpret_cast<const uint8_t *>(zero_chunk), *vs = ks;
        if (pg >= 0 && ch * 16 < D * es) {
          ks = kb + kv_k_off(a.kv, pg, ip) * es + ch * 16;
          vs = vb + kv_v_off(a.kv, pg, ip) * es + ch * 16;
        }
        if (FP8) {
          stage_k[i] = *reinterpret_cast<const u32x4 *>(ks);
          stage_v[i] = *reinterpret_cast<const u32x4 *>(vs);
        } else {
          const uint32_t at = uniform(lds_addr(dst + i * RPI * DP * 2));
          load_to_lds(ks, at);
          load_to_lds(vs, at + S::tile_bytes);
        }
      }
      return (uint64_t)__ballot(page >= 0);
    };
    auto store = [&](int buf) {  // FP8: the staged registers to LDS as bf16
#pragma unroll
      for (int i = 0; i < (FP8 ? LD : 0); ++i) {
        const int row = wave * own0 + i * RPI + lane_row(lane), q2 = 2 * (lane / RPI);
        uint8_t *dst = tiles + buf * 2 * S::tile_bytes + row * DP * 2;
        const int c0 = (q2 ^ swizzle<DP>(row)) * 16, c1 = ((q2 + 1) ^ swizzle<DP>(row)) * 16;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const u32x4 w = kv ? stage_v[i] : stage_k[i];
          const u32x4 w0 = {fp8_bf16_pair<false>(w.x), fp8_bf16_pair<true>(w.x), fp8_bf16_pair<false>(w.y), fp8_bf16_pair<true>(w.y)};
          const u32x4 w1 = {fp8_bf16_pair<false>(w.z), fp8_bf16_pair<true>(w.z), fp8_bf16_pair<false>(w.w), fp8_bf16_pair<true>(w.w)};
          *reinterpret_cast<u32x4 *>(dst + kv * S::tile_bytes + c0) = w0;
          *reinterpret_cast<u32x4 *>(dst + kv * S::tile_bytes + c1) = w1;
        }
      }
    };

    // Whether every row of the tile of rows sees all entries of the tile at j0.
    auto seen_by_all = [&](int j0) { return j0 >= t.lo_last && j0 + E <= min(t.hi_first, to); };
    // Where they do not, a value that is not finite must not meet the zero weight of a row that does not see it
    // (0 * inf): it is cleared in LDS, and added behind the loop to the rows that see it.  Whether there was one in
    // the rows that this wave stages.
    auto clear_odd = [&](int buf) {
      uint8_t *rows = tiles + buf * 2 * S::tile_bytes + S::tile_bytes + wave * own0 * DP * 2;
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < S::own * DP / 512; ++i) {
        const u32x4 w = reinterpret_cast<const u32x4 *>(rows)[i * 64 + lane];
#pragma unroll
        for (int y = 0; y < 4; ++y) any |= odd_bits(w[y]);
      }
      if (!__any(any != 0)) return false;
      uint32_t *v = reinterpret_cast<uint32_t *>(rows);
#pragma unroll 1
      for (int i = lane; i < S::own * DP / 2; i += 64) {
        const uint32_t e = odd_bits(v[i]);
        if (e) v[i] &= ~((e >> 15) * 0xffffu);
      }
      return true;
    };

    // ---- one tile of entries
    auto compute = [&](int j0, int buf, uint64_t paged) {
      const uint8_t *kt_base = tiles + buf * 2 * S::tile_bytes, *vt_base = kt_base + S::tile_bytes;
      f32x16 s[KT];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
        const int row = kt * 32 + c;
        const uint8_t *kr = kt_base + row * DP * 2;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const bf16x8 kf = *reinterpret_cast<const bf16x8 *>(kr + ((2 * ks + half) ^ swizzle<DP>(row)) * 16);
          s[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[ks], s[kt], 0, 0, 0);
        }
      }
      if (!seen_by_all(j0) || paged != kAll) {
        asm volatile("");   // (or the compiler makes selects of this, in every tile)
        // entries of registers i are 8 (i / 4) + i % 4 from the half's first
        const int at = j0 + 4 * half, lo_at = lo - at, hi_at = min(hi, to) - at;
        const uint64_t bits = paged >> (4 * half);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const uint32_t seen = seen_bits(lo_at - 32 * kt, hi_at - 32 * kt) & (uint32_t)(bits >> (32 * kt));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int keep = seen_sign(seen, i);
            s[kt][i] = __uint_as_float((__float_as_uint(s[kt][i]) & keep) | (0xff800000u & ~keep));
          }
        }
      }
      float mx = s[0][0];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kt][i]);
      mx = max_halves(mx) * cs;
      if (__any(mx > m + kSlack)) {  // true for the first visible entries (m = -inf)
        const float mn = fmaxf(m, mx);
        const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] *= f;
      }
      const float mu = m == -INFINITY ? 0.f : m;
      uint32_t p[KT][8];
      float sum = 0.f;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(s[kt][i], cs, -mu)), p1 = __builtin_amdgcn_exp2f(fmaf(s[kt][i + 1], cs, -mu));
          sum += p0;
          sum += p1;
          p[kt][i / 2] = f2bf16_pair(p0, p1);
        }
      l += sum;
      // transposing reads: lane i of 16 points at row i / 4, 4 dims i % 4, and gets dim i of 4 rows
      const int gq = lane >> 4, tr_row = 4 * (gq >> 1) + ((lane & 15) >> 2), tr_ch = 2 * (gq & 1) + ((lane & 3) >> 1),
                tr_off = 8 * (lane & 1);
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      auto values = [&](int row0, int d) {
        const int row = row0 + tr_row;
        const uint8_t *v = vt_base + row * DP * 2 + ((d * 4 + tr_ch) ^ swizzle<DP>(row)) * 16 + tr_off;
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)v));
      };
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          const u32x4 pw = {p[kt][4 * k2], p[kt][4 * k2 + 1], p[kt][4 * k2 + 2], p[kt][4 * k2 + 3]};
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const u32x2 v0 = values(kt * 32 + 16 * k2, d), v1 = values(kt * 32 + 16 * k2 + 8, d);
            const u32x4 vw = {v0.x, v0.y, v1.x, v1.y};
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vw), __builtin_bit_cast(bf16x8, pw), o[d], 0, 0, 0);
          }
        }
    };

    // ---- the loop: loads of the next tile run under the products of this one
    bool odd = false;
    if (TILE && j_first < to) {
      // NB - 1 tiles are under way before the loop (FP8: one, in registers), and one more is asked for in each turn,
      // into the buffer that the barrier has just freed
      constexpr int AHEAD = FP8 ? 1 : NB - 1;
      int buf = 0;
      uint64_t paged[AHEAD + 1] = {};
      peek(j_first);
#pragma unroll
      for (int x = 0; x < AHEAD; ++x) {
        if (x == 0 || j_first + x * step < to) paged[x] = issue(j_first + x * step, x);
        peek(j_first + (x + 1) * step);
      }
      for (int j0 = j_first; j0 < to; j0 += step) {
        if (FP8)
          store(buf);
        else if (AHEAD > 1 && j0 + (AHEAD - 1) * step < to)
          wait_loads<(AHEAD - 1) * 2 * LD>();
        else
          wait_loads<0>();
        __syncthreads();
        if (j0 + AHEAD * step < to) paged[AHEAD] = issue(j0 + AHEAD * step, (buf + AHEAD) % NB);
        peek(j0 + (AHEAD + 1) * step);
        if (t.tokens > 1 && !seen_by_all(j0)) {
          if (clear_odd(buf)) {
            odd = true;
            if (lane == 0) odd_sm = 1;
          }
          __syncthreads();
        }
        compute(j0, buf, paged[0] & kAll);
        buf = buf + 1 == NB ? 0 : buf + 1;
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) paged[x] = paged[x + 1];
      }
    }
    if (!TILE && j_first < to) {
      int buf = 0;
      peek(j_first);
      uint64_t paged = issue(j_first, 0);
      peek(j_first + step);
      if (FP8) store(0);
      for (int j0 = j_first; j0 < to; j0 += step) {
        const bool more = j0 + step < to;
        uint64_t paged_next = 0;
        if (more) {
          paged_next = issue(j0 + step, NB == 2 ? buf ^ 1 : 0);
          if (!FP8) wait_loads<2 * LD>();
        } else if (!FP8) {
          wait_loads<0>();
        }
        peek(j0 + 2 * step);
        const int at = NB == 2 ? buf : 0;
        if (t.tokens > 1 && !seen_by_all(j0)) odd |= clear_odd(at);
        compute(j0, at, paged & kAll);
        if (FP8 && more) store(0);
        buf ^= 1;
        paged = paged_next;
      }
    }
    if (TILE) {
      __syncthreads();
      odd = odd_sm != 0;
    }
    if (odd) {
      // the cleared values, entry by entry, with the weights formed anew: m is the final maximum
#pragma unroll 1
      for (int j0 = j_first; j0 < to; j0 += step) {
        if (seen_by_all(j0)) continue;
#pragma unroll 1
        for (int j = max(j0, t.lo); j < min(j0 + E, to); ++j) {
          int in_page;
          const int page = kv_page(a.kv, table, shift, j, &in_page);
          if (page < 0) continue;
          const uint8_t *vp = vb + kv_v_off(a.kv, page, in_page) * es, *kp = kb + kv_k_off(a.kv, page, in_page) * es;
          bool any = false;
          for (int d = lane; d < D; d += 64) {
            const uint32_t v = FP8 ? vp[d] : reinterpret_cast<const uint16_t *>(vp)[d];
            any |= FP8 ? (v & 0x7f) == 0x7f : (v & 0x7f80) == 0x7f80;
          }
          if (!__any(any)) continue;
          float dot = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            if (ks * 16 < D) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int d = 16 * ks + 8 * half + e;
                dot = fmaf((float)q[ks][e], FP8 ? e4m3_pair<false>(kp[d]).x : bf16f(reinterpret_cast<const uint16_t *>(kp)[d]), dot);
              }
            }
          const float w = __builtin_amdgcn_exp2f(fmaf(sum_halves(dot), cs, -m));
          if (j < lo || j >= hi) continue;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int dim = d * 32 + 8 * (i / 4) + 4 * half + i % 4;
              if (dim < D) {
                const float v = FP8 ? e4m3_pair<false>(vp[dim]).x : bf16f(reinterpret_cast<const uint16_t *>(vp)[dim]);
                if (!(fabsf(v) < INFINITY)) o[d][i] = fmaf(w, v, o[d][i]);
              }
            }
        }
      }
    }

    // ---- results
    l = sum_halves(l);
    if (TILE) {
      if (!row_live) return;
      const int64_t rh = (int64_t)row_t * a.q_heads + row_h;
      if (direct) {
        const float inv = l == 0.f ? 0.f : a.kv.v_scale / l;
        uint16_t *op = a.out.p + row_t * a.out.row + row_h * a.out.head + 4 * half;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            if (d * 32 + 2 * i < D) {
              const u32x2 w = {f2bf16_pair(o[d][i] * inv, o[d][i + 1] * inv), f2bf16_pair(o[d][i + 2] * inv, o[d][i + 3] * inv)};
              *reinterpret_cast<u32x2 *>(op + d * 32 + 2 * i) = w;
            }
        if (a.lse && half == 0) a.lse[rh] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
      } else {
        const int64_t at = (int64_t)split * a.n * a.q_heads + rh;
        float *op = part_sums<TILE>(a, plan, at) + 4 * half;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            if (d * 32 + 2 * i < D) *reinterpret_cast<f32x4 *>(op + d * 32 + 2 * i) = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
        if (half == 0) *part_stats<TILE>(a, at) = make_float2(m, l);
      }
      return;
    }
    // SPLIT: join the waves
    __syncthreads();  // every wave is done with its tiles
    float *jo = reinterpret_cast<float *>(sm);                 // [waves][32][DP]
    constexpr int JS = 32 * DP;
    {
      float *mine = jo + wave * JS + c * DP + 4 * half;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<f32x4 *>(mine + d * 32 + 2 * i) = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
      if (half == 0) {
        jm[wave][c] = m;
        jl[wave][c] = l;
      }
      if (wave == 0 && half == 0) {
        j_row[c] = row_t;
        j_head[c] = row_h;
      }
    }
    __syncthreads();
    for (int it = threadIdx.x; it < t.tokens * G * (DP / 4); it += S::waves * 64) {
      const int jr = it / (DP / 4), d4 = it % (DP / 4) * 4;
      if (d4 >= D) continue;
      const int rt = j_row[jr], rh_ = j_head[jr];
      float mm = jm[0][jr];
#pragma unroll
      for (int w = 1; w < S::waves; ++w) mm = fmaxf(mm, jm[w][jr]);
      float ll = 0.f;
      f32x4 s4 = {0.f, 0.f, 0.f, 0.f};
      const float mu = mm == -INFINITY ? 0.f : mm;   // no maximum: nothing was seen (sums of 0), or NaN alone (NaN)
#pragma unroll
      for (int w = 0; w < S::waves; ++w) {
        const float f = __builtin_amdgcn_exp2f(jm[w][jr] - mu);
        ll = fmaf(jl[w][jr], f, ll);
        const f32x4 v = *reinterpret_cast<const f32x4 *>(jo + w * JS + jr * DP + d4);
#pragma unroll
        for (int y = 0; y < 4; ++y) s4[y] = fmaf(v[y], f, s4[y]);
      }
      if (direct) {
        const float inv = ll == 0.f ? 0.f : a.kv.v_scale / ll;
        const u32x2 w = {f2bf16_pair(s4[0] * inv, s4[1] * inv), f2bf16_pair(s4[2] * inv, s4[3] * inv)};
        *reinterpret_cast<u32x2 *>(a.out.p + rt * a.out.row + rh_ * a.out.head + d4) = w;
        if (a.lse && d4 == 0) a.lse[(int64_t)rt * a.q_heads + rh_] = ll == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
      } else {
        const int64_t at = (blockIdx.x * 2ll + (x == 0)) * 32 + jr;
        *reinterpret_cast<f32x4 *>(part_sums<TILE>(a, plan, at) + d4) = s4;
        if (d4 == 0) *part_stats<TILE>(a, at) = make_float2(mm, ll);
      }
    }
    if (unit < unit_end) __syncthreads();  // before the next pair's tiles
  } while (!TILE && unit < unit_end);
}

// Joins the parts of a row, in their order.  One workgroup of 4 waves per (row, head): wave w
// adds parts w, w + 4, ...; lane i holds dims 4 i .. 4 i + 3.
template <bool TILE>
__global__ __launch_bounds__(256) void attn_merge_kernel(AttnArgs a, Plan plan) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  __shared__ f32x4 so[4][64];
  __shared__ float sl[4];
  const int row = blockIdx.x / a.q_heads, h = blockIdx.x - row * a.q_heads, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int G = a.q_heads / a.kv.kv_heads, g = h / G;
  // the sequence of this row, then its tile and where its parts are
  Tile t;
  t.b = -1;
  int before = 0, total = 0, start = 0;
  for (int b0 = 0; b0 < a.kv.batch; b0 += 64) {
    int first, rows, len;
    lane_sequence(a, b0, &first, &rows, &len);
    const int mine = TILE ? 0 : sequence_units(a, plan, rows, len), upto = before + scan64(mine);
    const uint64_t hit = __ballot(row >= first && row < first + rows);
    if (hit && t.b < 0) {
      const int w = uniform(__builtin_ctzll(hit));
      take_sequence(t, b0, w, first, rows, len);
      start = lane_value(upto - mine, w);
      if (TILE) break;
    }
    before = lane_value(upto, 63);
  }
  total = before;
  if (t.b < 0) return;
  const int own_t0 = (row - t.first) / plan.tile_tokens * plan.tile_tokens;
  if (!TILE)
    for (t.t0 = 0; t.t0 < own_t0; t.t0 += plan.tile_tokens) {
      tile_entries(a, plan, t);
      start += (kBegin + t.parts) * a.kv.kv_heads;
    }
  t.t0 = own_t0;
  tile_entries(a, plan, t);
  int parts = t.parts, b_first = 0;
  int64_t at0 = (int64_t)row * a.q_heads + h, stride = (int64_t)a.n * a.q_heads;   // TILE: part s at at0 + s * stride
  if (!TILE) {
    const int share = max(1, unit_share(plan, total));
    start += g * (kBegin + t.parts) + kBegin;
    b_first = start / share;
    parts = (start + t.parts - 1) / share - b_first + 1;
    at0 = b_first * 64ll + (row - t.first - t.t0) * G + h - g * G;   // part 0 begins a pair: place 1; the others 0
    stride = 64;
  }
  if (parts == 1) return;  // written by its workgroup
  if (!TILE && (b_first < 0 || parts < 1 || b_first + (int64_t)parts > plan.blocks)) return;   // as in find_unit
  auto place = [&](int s) { return at0 + s * stride + (!TILE && s == 0 ? 32 : 0); };
  float mm = -INFINITY;
  for (int s = lane; s < parts; s += 64) mm = fmaxf(mm, part_stats<TILE>(a, place(s))->x);
  for (int d = 32; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor(mm, d, 64));
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  float ll = 0.f;
  const bool live = 4 * lane < a.kv.head_dim;
  const float mu = mm == -INFINITY ? 0.f : mm;   // as where the waves are joined
#pragma unroll 4
  for (int s = wave; s < parts; s += 4) {
    const float2 st = *part_stats<TILE>(a, place(s));
    const float f = __builtin_amdgcn_exp2f(st.x - mu);
    ll = fmaf(st.y, f, ll);
    if (live) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(part_sums<TILE>(a, plan, place(s)) + 4 * lane);
#pragma unroll
      for (int y = 0; y < 4; ++y) sum[y] = fmaf(v[y], f, sum[y]);
    }
  }
  so[wave][lane] = sum;
  if (lane == 0) sl[wave] = ll;
  __syncthreads();
  if (wave) return;
  ll = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  const float inv = ll == 0.f ? 0.f : a.kv.v_scale / ll;
  if (live) {
    f32x4 v;
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] = ((so[0][lane][y] + so[1][lane][y]) + (so[2][lane][y] + so[3][lane][y])) * inv;
    const u32x2 w = {f2bf16_pair(v[0], v[1]), f2bf16_pair(v[2], v[3])};
    *reinterpret_cast<u32x2 *>(a.out.p + row * a.out.row + h * a.out.head + 4 * lane) = w;
  }
  if (a.lse && lane == 0) a.lse[(int64_t)row * a.q_heads + h] = ll == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
}

// ------------------------------------------------------------------ weigh
// The weights that entries receive: S^T = K Q^T once more, with the row's log-sum-exp known.
// A workgroup goes over the rows that see any of its 128 entries, 64 RG at a time, from LDS.  Wave
// (e, x) keeps the keys of 32 entries in registers (A operand) and takes 64 of the rows:
// a lane adds up the weights of its rows (columns) for 16 entries, and the sums of the lanes and
// of the RG waves are joined through LDS at the end.  No two workgroups share an entry, so
// nothing is added atomically.  Bound by the exponentials (one
// for each entry, row pair, with a multiply-add and an add) rather than by the product.
// (8111 entries of 8 heads, 1000 new tokens: with one wave for 32 entries 196 us, with two 125; with two shorter
// sequences beside it, 2029 tokens in all, 144.)  While a CU is busy its
// SIMDs issue vector or matrix instructions all the time, 3 : 1.  Products of the next rows between the exponentials of
// these, four tiles of rows under way, or the sequences with most rows first did not help (143 -> 166, 194, 187 us).
constexpr int RG = 2;
template <int DP>
struct WeighShape {
  static constexpr int entries = 4 * 32, rows = 64 * RG, threads = 256 * RG;
  static constexpr int tile_bytes = rows * DP * 2;
};

template <int DP, bool FP8>
__global__ __launch_bounds__(256 * RG, DP == 64 ? 4 : 2) void weigh_kernel(AttnArgs a) {
  using S = WeighShape<DP>;
  constexpr int KS = DP / 16, CPR = DP / 8, RPI = 64 / CPR, LD = 16 / RPI;
  __shared__ __attribute__((aligned(16))) uint8_t sm[2 * S::tile_bytes > RG * 128 * 33 * 4 ? 2 * S::tile_bytes : RG * 128 * 33 * 4];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 31, half = lane >> 5;
  const int D = a.kv.head_dim, G = a.q_heads / a.kv.kv_heads;
  int id = blockIdx.x;
  const int g = id % a.kv.kv_heads;
  id /= a.kv.kv_heads;
  // then the sequences, then the entries: a sequence's first entries, which most rows see, start first
  const int e0 = id / a.kv.batch * S::entries, b = id - e0 / S::entries * a.kv.batch;
  bool bad = false;
  const int len = kv_len(a.kv, a.kv.len[b], &bad);
  int first;
  const int rows = kv_rows(a.q_start[b], a.q_start[b + 1], a.n, &first, &bad);
  if (bad) raise_status(a.kv);
  if (e0 >= len || rows == 0) return;
  // tokens that see an entry of the workgroup: at >= e0, and at < last entry + window
  const int before = len - rows, e1 = min(e0 + S::entries, len);
  const int i0 = max(0, e0 - before);
  const int i1 = a.window > 0 ? (int)min((int64_t)rows, (int64_t)e1 - 1 + a.window - before) : rows;
  if (i0 >= i1) return;
  // keys of this wave
  const int ew = e0 + (wave & 3) * 32, rw = (wave >> 2) * 64;
  bf16x8 key[KS];
  uint32_t paged;
  {
    const int j = ew + c;
    int ip = 0, page = -1;
    if (j < len) {
      page = kv_page(a.kv, a.kv.table + b * a.kv.table_stride, a.shift, j, &ip);
      if (page < 0) raise_status(a.kv);
    }
    paged = (uint32_t)__ballot(page >= 0);
    const int64_t off = kv_k_off(a.kv, max(page, 0), ip) + a.kv.k_head * g + 8 * half;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      u32x4 w = {0, 0, 0, 0};
      if (page >= 0 && ks * 16 < D) {
        if (FP8) {
          const u32x2 v = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(a.kv.k) + off + 16 * ks);
          w = u32x4{fp8_bf16_pair<false>(v.x), fp8_bf16_pair<true>(v.x), fp8_bf16_pair<false>(v.y), fp8_bf16_pair<true>(v.y)};
        } else {
          w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.kv.k) + off + 16 * ks);
        }
      }
      key[ks] = __builtin_bit_cast(bf16x8, w);
    }
  }
  // whether a product with a row of zeros may not be 0: a key that is not finite
  uint32_t odd_key = 0;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const u32x4 w = __builtin_bit_cast(u32x4, key[ks]);
#pragma unroll
    for (int y = 0; y < 4; ++y) odd_key |= odd_bits(w[y]);
  }
  const bool odd_keys = __any(odd_key != 0);
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  const float cs = a.scale * a.kv.k_scale * kLog2e;

  // A tile holds the G heads of T = 64 RG / G tokens, so a lane's (token, head) within it is the same in every tile:
  // its addresses are a scalar base and a constant offset.  Rows of LDS past T G stay zero.
  const int T = S::rows / G;
  // rows to LDS: wave w stages rows 16 w .. 16 w + 15
  uint32_t st_off[LD];
  int st_tok[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int row = 16 * wave + i * RPI + lane / CPR, ch = (lane % CPR) ^ swizzle<DP>(row), tok = row / G;
    st_off[i] = (uint32_t)((tok * a.q.row + (g * G + row - tok * G) * a.q.head + ch * 8) * 2);
    st_tok[i] = ch * 8 < D ? tok : 1 << 30;   // chunks behind head_dim: never a token
  }
  const bool near = 129 * a.q.row + (int64_t)a.q_heads * a.q.head < (1ll << 31);   // offsets of 32 bits do
  int ls_tok[2];
  uint32_t ls_off[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = rw + 32 * x + c;
    ls_tok[x] = row / G;
    ls_off[x] = ls_tok[x] * a.q_heads + g * G + row - ls_tok[x] * G;
    if (row >= T * G) ls_tok[x] = 1 << 30;
  }
#pragma unroll
  for (int i = 0; i < 2 * S::tile_bytes / 16 / S::threads; ++i) *reinterpret_cast<u32x4 *>(sm + (i * S::threads + threadIdx.x) * 16) = u32x4{0, 0, 0, 0};
  __syncthreads();
  auto issue = [&](int i, int buf) {  // the tile from token i on
    const uint16_t *base = a.q.p + (int64_t)(first + i) * a.q.row;
#pragma unroll
    for (int x = 0; x < LD; ++x) {
      const uint32_t lds = uniform(lds_addr(sm + buf * S::tile_bytes + (16 * wave + x * RPI) * DP * 2));
      if (near && i + T <= i1) {
        if (st_tok[x] < T) load_to_lds(base, st_off[x], lds);
      } else {  // a last tile with fewer tokens: zeros behind them
        const int row = 16 * wave + x * RPI + lane / CPR, ch = (lane % CPR) ^ swizzle<DP>(row), tok = row / G;
        const uint16_t *src = base + tok * a.q.row + (g * G + row - tok * G) * a.q.head + ch * 8;
        if (st_tok[x] >= T || i + st_tok[x] >= i1) src = reinterpret_cast<const uint16_t *>(zero_chunk);
        load_to_lds(src, lds);
      }
    }
  };
  float lse[2];
  auto next_lse = [&](int i) {  // +inf behind the rows: exp(-inf) = 0
    const float *base = a.lse + (int64_t)(first + i) * a.q_heads;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool in = i + ls_tok[x] < i1;
      const float v = base[in ? ls_off[x] : 0];
      lse[x] = in ? v : INFINITY;
    }
  };
  next_lse(i0);
  issue(i0, 0);
  int buf = 0;
  for (int i = i0; i < i1; i += T) {
    wait_loads<0>();
    __syncthreads();
    float l2[2] = {lse[0] * kLog2e, lse[1] * kLog2e};
    asm volatile("" : "+v"(l2[0]), "+v"(l2[1]));   // here, before the next loads, or it waits for them
    if (i + T < i1) {
      next_lse(i + T);
      issue(i + T, buf ^ 1);
    }
    f32x16 s[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[x][e] = 0.f;
    const uint8_t *qr = sm + buf * S::tile_bytes + (rw + c) * DP * 2;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int at = ((2 * ks + half) ^ swizzle<DP>(c)) * 16;   // rows c and c + 32 have one swizzle
#pragma unroll
      for (int x = 0; x < 2; ++x)
        s[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key[ks], *reinterpret_cast<const bf16x8 *>(qr + x * 32 * DP * 2 + at), s[x], 0, 0, 0);
    }
    // every row of this tile sees every entry of the wave, and all entries have pages: no masks.  (But for rows that add
    // nothing whatever their scores, and rows of zeros beside a key that is not finite: 0 inf and inf - inf are NaN.)
    const int last_tok = min(i + T, i1) - 1;
    if (before + i >= ew + 31 && (a.window == 0 || before + last_tok - a.window < ew) && paged == ~0u && !odd_keys &&
        !__any(fminf(l2[0], l2[1]) == -INFINITY)) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[e] += __builtin_amdgcn_exp2f(fmaf(s[0][e], cs, -l2[0])) + __builtin_amdgcn_exp2f(fmaf(s[1][e], cs, -l2[1]));
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        asm volatile("");   // (or the compiler makes selects of this, in every tile)
        int lo = 0, hi = 0;
        if (i + ls_tok[x] < i1 && l2[x] != -INFINITY) kv_seen(len, rows, i + ls_tok[x], a.window, &lo, &hi);
        const uint32_t seen = seen_bits(lo - ew - 4 * half, hi - ew - 4 * half) & (paged >> (4 * half));
#pragma unroll
        for (int y = 0; y < 16; ++y)
          acc[y] += __uint_as_float(__float_as_uint(__builtin_amdgcn_exp2f(fmaf(s[x][y], cs, -l2[x]))) & seen_sign(seen, y));
      }
    }
    buf ^= 1;
  }
  // join the rows: 32 entries x 32 columns (padded) of every wave
  float *join = reinterpret_cast<float *>(sm);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) join[(wave * 32 + 8 * (i / 4) + 4 * half + i % 4) * 33 + c] = acc[i];
  __syncthreads();
  if (wave >= 4) return;
  float sum = 0.f;   // lane (c, half): entry c, columns 16 half .. + 15 of its RG waves
#pragma unroll
  for (int x = 0; x < 16; ++x)
#pragma unroll
    for (int y = 0; y < RG; ++y) sum += join[((wave + 4 * y) * 32 + c) * 33 + 16 * half + x];
  sum = sum_halves(sum);
  const int j = ew + c;
  if (half == 0 && j < len && ((paged >> c) & 1)) a.acc[((int64_t)b * a.kv.kv_heads + g) * a.acc_stride + j] += sum;
}

// The same for few rows a pair (decode steps): a wave takes 32 entries by itself, with its rows, 32 at a time,
// straight from global memory (every wave of the pair reads the same few); no barrier.  Units of 128 entries are
// shared out over a fixed number of workgroups, since the start of a workgroup costs some 4 ns of the launch: a grid
// over (sequence, head, 128 entries of the table's width) took 20 us for 16 sequences of up to 8192 entries, most of
// it workgroups without entries.
constexpr int kFewBlocks = 512;

template <int DP, bool FP8>
__global__ __launch_bounds__(256, DP == 256 ? 2 : 4) void weigh_few_kernel(AttnArgs a) {
  constexpr int KS = DP / 16;
  __shared__ float join_sm[4][32 * 33];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 31, half = lane >> 5;
  const int D = a.kv.head_dim, G = a.q_heads / a.kv.kv_heads;
  const float cs = a.scale * a.kv.k_scale * kLog2e;
  const int T = 32 / G, tok = c / G;
  // units of the lane's sequence of the first 64, and their running sum
  auto units = [&](int rows, int len) { return rows > 0 ? (len + 127) / 128 * a.kv.kv_heads : 0; };
  Tile t;
  int first, rows, len;
  lane_sequence(a, 0, &first, &rows, &len);
  const int mine0 = units(rows, len), upto0 = scan64(mine0), first0 = first, rows0 = rows, len0 = len;
  int total = lane_value(upto0, 63);
  for (int b0 = 64; b0 < a.kv.batch; b0 += 64) {
    lane_sequence(a, b0, &first, &rows, &len);
    total += lane_value(scan64(units(rows, len)), 63);
  }
  const int share = (total + gridDim.x - 1) / gridDim.x;
  const int u1 = (int)min((int64_t)total, ((int64_t)blockIdx.x + 1) * share);
  int g = a.kv.kv_heads, e = 0;
  t.len = 0;
  for (int u = min((int64_t)total, (int64_t)blockIdx.x * share); u < u1; ++u) {
    e += 128;
    if (e >= t.len) {   // the next head, or the next sequence
      e = 0;
      if (++g >= a.kv.kv_heads) {
        int before = 0;
        for (int b0 = 0; b0 < a.kv.batch; b0 += 64) {
          int mine = mine0, upto = upto0;
          first = first0, rows = rows0, len = len0;
          if (b0) {
            lane_sequence(a, b0, &first, &rows, &len);
            mine = units(rows, len);
            upto = before + scan64(mine);
          }
          const uint64_t hit = __ballot(upto > u && upto - mine <= u);
          if (hit) {
            const int w = uniform(__builtin_ctzll(hit));
            take_sequence(t, b0, w, first, rows, len);
            const int left = u - lane_value(upto - mine, w), per = (t.len + 127) / 128;
            g = left / per;
            e = (left - g * per) * 128;
            break;
          }
          before = lane_value(upto, 63);
        }
      }
    }
    const int ew = e + wave * 32, before = t.len - t.rows;
    if (ew >= t.len) continue;
    const int i0 = max(0, ew - before);
    const int i1 = a.window > 0 ? (int)min((int64_t)t.rows, (int64_t)min(ew + 32, t.len) - 1 + a.window - before) : t.rows;
    if (i0 >= i1) continue;
    const int head = g * G + c - tok * G;
    u32x4 key[KS];   // FP8: 8 bytes of each
    uint32_t paged;
    {
      const int j = ew + c;
      int ip = 0, page = -1;
      if (j < t.len) {
        page = kv_page(a.kv, a.kv.table + t.b * a.kv.table_stride, a.shift, j, &ip);
        if (page < 0) raise_status(a.kv);
      }
      paged = (uint32_t)__ballot(page >= 0);
      const int64_t off = kv_k_off(a.kv, max(page, 0), ip) + a.kv.k_head * g + 8 * half;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        key[ks] = u32x4{0, 0, 0, 0};
        if (page >= 0 && ks * 16 < D) {
          if (FP8) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(a.kv.k) + off + 16 * ks);
            key[ks].x = v.x;
            key[ks].y = v.y;
          } else {
            key[ks] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.kv.k) + off + 16 * ks);
          }
        }
      }
    }
    float acc[16];
#pragma unroll
    for (int y = 0; y < 16; ++y) acc[y] = 0.f;
    for (int i = i0; i < i1; i += T) {
      const bool in = tok < T && i + tok < i1;
      const int row = t.first + i + (in ? tok : 0), h = in ? head : g * G;   // others: another row's, and masked
      const float lse = a.lse[(int64_t)row * a.q_heads + h];
      const uint16_t *qp = a.q.p + row * a.q.row + h * a.q.head + 8 * half;
      u32x4 q[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) q[ks] = *reinterpret_cast<const u32x4 *>(qp + (ks * 16 < D ? 16 * ks : 0));
      f32x16 s;
#pragma unroll
      for (int y = 0; y < 16; ++y) s[y] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        u32x4 w = key[ks];
        if (FP8) w = u32x4{fp8_bf16_pair<false>(w.x), fp8_bf16_pair<true>(w.x), fp8_bf16_pair<false>(w.y), fp8_bf16_pair<true>(w.y)};
        if (ks * 16 < D)
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, q[ks]), s, 0, 0, 0);
      }
      int lo = 0, hi = 0;
      if (in && lse != -INFINITY) kv_seen(t.len, t.rows, i + tok, a.window, &lo, &hi);
      const uint32_t seen = seen_bits(lo - ew - 4 * half, hi - ew - 4 * half) & (paged >> (4 * half));
      const float l2 = lse * kLog2e;
#pragma unroll
      for (int y = 0; y < 16; ++y)
        acc[y] += __uint_as_float(__float_as_uint(__builtin_amdgcn_exp2f(fmaf(s[y], cs, -l2))) & seen_sign(seen, y));
    }
    float *join = join_sm[wave];   // the wave's own: its LDS operations run in order
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int y = 0; y < 16; ++y) join[(8 * (y / 4) + 4 * half + y % 4) * 33 + c] = acc[y];
    __builtin_amdgcn_wave_barrier();
    float sum = 0.f;
#pragma unroll
    for (int y = 0; y < 16; ++y) sum += join[c * 33 + 16 * half + y];
    sum = sum_halves(sum);
    const int j = ew + c;
    if (half == 0 && j < t.len && ((paged >> c) & 1)) a.acc[((int64_t)t.b * a.kv.kv_heads + g) * a.acc_stride + j] += sum;
  }
}

bool split_shape(const oes_kv &kv, int q_heads, int n) {
  // SPLIT holds 32 rows; beyond, on average per sequence and cache head, TILE's 128 fill up better
  const int G = q_heads / kv.kv_heads;
  return G <= 32 && (int64_t)n * G <= 32ll * kv.batch;
}

int head_pad(const oes_kv &kv) { return kv.head_dim <= 64 ? 64 : (kv.head_dim <= 128 ? 128 : 256); }

Plan make_plan(const oes_kv &kv, int q_heads, int n) {
  const int G = q_heads / kv.kv_heads, dp = head_pad(kv);
  const bool split = split_shape(kv, q_heads, n), fp8 = kv.elem == OES_ELEM_E4M3;
  Plan p = {};
  p.chunk_log = -1;
  p.tile_tokens = (split ? 32 : 128) / G;
  // every sequence with rows has at most one tile that is not full
  const int64_t tiles = std::min<int64_t>(n, ((int64_t)n + (int64_t)kv.batch * (p.tile_tokens - 1)) / p.tile_tokens);
  p.tiles = (int)tiles;
  const int64_t cap = ((int64_t)kv.max_pages * kv.page_size + 31) / 32 * 32 + 32;   // entries of a tile, from its base
  if (split) {
    p.chunk_log = dp == 256 ? 6 : 7;   // 32 entries a wave
    p.chunk = 1 << p.chunk_log;
    // as many workgroups as are resident at once: LDS holds two to a CU, or one of the bf16 cache's 128 KiB
    p.blocks = (int)std::min<int64_t>(dp == 64 || (fp8 && dp == 128) ? 512 : 256, tiles * kv.kv_heads * (kBegin + (cap + p.chunk - 1) / p.chunk));
    p.splits = cap <= p.chunk ? 1 : 2;
  } else {
    const int64_t parts = std::max<int64_t>(1, 512 / (tiles * kv.kv_heads));
    int64_t chunk = std::max<int64_t>(256, ((cap + parts - 1) / parts + 63) / 64 * 64);
    p.splits = (int)((cap + chunk - 1) / chunk);
    if (p.splits == 1) chunk = cap;
    p.chunk = (int)std::min<int64_t>(chunk, 1 << 30);
  }
  return p;
}

template <int DP, bool FP8, bool TILE>
hipError_t launch_shape(const AttnArgs &a, const Plan &p, uint32_t blocks, hipStream_t s) {
  hipLaunchKernelGGL((attn_kernel<DP, FP8, TILE>), dim3(blocks), dim3(Shape<DP, FP8, TILE>::waves * 64), 0, s, a, p);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_dim(const AttnArgs &a, const Plan &p, bool split, uint32_t blocks, hipStream_t s) {
  if (a.kv.elem == OES_ELEM_E4M3) return split ? launch_shape<DP, true, false>(a, p, blocks, s) : launch_shape<DP, true, true>(a, p, blocks, s);
  return split ? launch_shape<DP, false, false>(a, p, blocks, s) : launch_shape<DP, false, true>(a, p, blocks, s);
}

}  // namespace

bool attn_fits(const oes_kv &kv, int q_heads, int n) {
  const Plan p = make_plan(kv, q_heads, n);
  const bool split = split_shape(kv, q_heads, n);
  const int64_t cap = (int64_t)kv.max_pages * kv.page_size, rows = (int64_t)n * q_heads;
  return launch_fits(split ? p.blocks : (int64_t)p.tiles * kv.kv_heads * p.splits, 256) &&
         (p.splits == 1 ? rows <= 0x7fffffff : launch_fits(rows, 256)) &&
         (int64_t)p.tiles * kv.kv_heads * (cap / 64 + 2 + kBegin) <= 0x7fffffff;   // units, counted in 32 bits
}

int64_t attn_workspace_bytes(const oes_kv &kv, int q_heads, int n) {
  const Plan p = make_plan(kv, q_heads, n);
  if (p.splits == 1) return 0;
  const int64_t rows = split_shape(kv, q_heads, n) ? (int64_t)p.blocks * 64 : (int64_t)p.splits * n * q_heads;
  return rows * (kv.head_dim + 2) * 4;
}

hipError_t launch_attn(const AttnArgs &args, hipStream_t s) {
  AttnArgs a = args;
  a.shift = kv_shift(a.kv.page_size);
  const Plan p = make_plan(a.kv, a.q_heads, a.n);
  const bool split = split_shape(a.kv, a.q_heads, a.n);
  const int64_t blocks = split ? p.blocks : (int64_t)p.tiles * a.kv.kv_heads * p.splits;
  const int dp = head_pad(a.kv);
  const hipError_t e = dp == 64 ? launch_dim<64>(a, p, split, (uint32_t)blocks, s)
                                : (dp == 128 ? launch_dim<128>(a, p, split, (uint32_t)blocks, s) : launch_dim<256>(a, p, split, (uint32_t)blocks, s));
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 g((uint32_t)(a.n * a.q_heads)), b(256);
  if (split)
    hipLaunchKernelGGL(attn_merge_kernel<false>, g, b, 0, s, a, p);
  else
    hipLaunchKernelGGL(attn_merge_kernel<true>, g, b, 0, s, a, p);
  return hipGetLastError();
}

namespace {
// 128 entries each of every cache head, over the tables' width
int64_t weigh_units(const oes_kv &kv) { return ((int64_t)kv.max_pages * kv.page_size + 127) / 128 * kv.kv_heads * kv.batch; }

template <int DP, bool FP8>
hipError_t launch_weigh(const AttnArgs &a, hipStream_t s) {
  const bool few = split_shape(a.kv, a.q_heads, a.n);
  const int64_t blocks = weigh_units(a.kv);
  if (few)
    hipLaunchKernelGGL((weigh_few_kernel<DP, FP8>), dim3((uint32_t)std::min<int64_t>(blocks, kFewBlocks)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((weigh_kernel<DP, FP8>), dim3((uint32_t)blocks), dim3(512), 0, s, a);
  return hipGetLastError();
}
}  // namespace

bool attn_weigh_fits(const oes_kv &kv, int q_heads, int n) {
  // (decode steps: units are counted in 32 bits)
  return (split_shape(kv, q_heads, n) ? weigh_units(kv) <= 0x7fffffff : launch_fits(weigh_units(kv), 512)) &&
         (int64_t)n * q_heads <= 0x7fffffff;
}

hipError_t launch_attn_weigh(const AttnArgs &args, hipStream_t s) {
  AttnArgs a = args;
  a.shift = kv_shift(a.kv.page_size);
  const bool fp8 = a.kv.elem == OES_ELEM_E4M3;
  if (a.kv.head_dim <= 64) return fp8 ? launch_weigh<64, true>(a, s) : launch_weigh<64, false>(a, s);
  if (a.kv.head_dim <= 128) return fp8 ? launch_weigh<128, true>(a, s) : launch_weigh<128, false>(a, s);
  return fp8 ? launch_weigh<256, true>(a, s) : launch_weigh<256, false>(a, s);
}

}  // namespace oes
