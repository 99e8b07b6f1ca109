// Shared pieces of the attention kernels (forward, backward, single token).
//
// Query i of a sequence stands at position pos = i + (keys - queries) and
// sees key j when j <= pos and (j > pos - window or j < sinks).
//
// Matrix products run on v_mfma_f32_32x32x16_bf16 (A 32 x 16, B 16 x 32):
//   A: lane l holds row l & 31, B: column l & 31, each with the 8 reduction
//   places of half h = l >> 5; D: lane l holds column l & 31 and rows
//   8 (r >> 2) + 4 h + (r & 3) for r = 0 .. 15.
// A score block is computed so that its columns are what the next product
// keeps as columns (queries in the forward pass and for dQ, keys for dK and
// dV). Then 8 consecutive values of a lane, rounded to bf16, are at once the
// B fragment of a 16-deep product over the block's rows, at the rows
// 4 h + 0..3 and 8 + 4 h + 0..3 (+ 16): no value changes lanes. The A
// fragment of that product takes the same rows in the same order from an
// LDS tile [row][D] by the transposing read ds_read_b64_tr_b16.
//
// That rounding of probabilities (and of dS) to bf16 is the one the matrix
// instructions ask for, at twice the rate of any wider type or better: each is
// off by at most 2^-8 of itself, independently, and the products and all sums
// stay float32. Sums of probabilities take them before the rounding. (Single
// tokens, which wait for memory, take the remainder in a second product.)
#pragma once

#include "launch.hpp"

namespace qlora {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) void gbl_void_t;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s_t;

constexpr float kAttnLog2e = 1.4426950408889634f;

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
  return f32x16{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}
__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Lanes l and l + 32 hold the two halves of a query's (or key's) rows.
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16-byte chunk c of row R of an LDS tile with DP elements per row is stored
// at chunk c ^ tile_swz(R). It spreads every kind of fragment read over the
// 64 banks: 16-byte reads of 32 rows at one chunk or of 16 rows at 4 chunks
// (the hardware serves lanes 0-3, 12-15, 20-23, 24-27 together, then the other
// half of 32), and transposing reads of 4 rows at 4 neighbouring chunks or of
// 8 rows at 2. No conflicts are counted.
template <int DP>
__device__ __forceinline__ constexpr int tile_swz(int R) {
  const int b2 = (R >> 2) & 1, b3 = (R >> 3) & 1;
  const int low = (b2 ^ b3) << 1 | b3;
  return DP == 128 ? ((R & 3) << 2) | low : (((R >> 1) & 1) << 2) | low;
}

// LDS-DMA of 64 rows x DP elements by the NW waves of a workgroup; row r of the
// tile is row min(r, last) of `src` (byte pitch `pitch`), so no row past the
// sequence is touched. A wave's instruction i brings 64 / CH rows; chunks past
// D repeat the last one (their products meet zeros in the other operand, or
// columns that are not stored).
template <int DP, int NW>
struct TileLoad {
  static constexpr int CH = DP / 8;           // chunks per row
  static constexpr int RPI = 64 / CH;         // rows per instruction
  static constexpr int NI = 64 / (NW * RPI);  // instructions per wave
  uint32_t off[NI];                           // of this lane's 16 bytes, from the tile's first row
  uint32_t pitch;
  int r0;  // this lane's row in the first instruction

  __device__ __forceinline__ TileLoad(int64_t pitch_elements, int D, int w, int l) {
    pitch = 2u * (uint32_t)pitch_elements;
    r0 = w * NI * RPI + l / CH;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = r0 + i * RPI;
      off[i] = (uint32_t)r * pitch + 16u * min((l % CH) ^ tile_swz<DP>(r), D / 8 - 1);
    }
  }
  __device__ __forceinline__ void operator()(const uint16_t* src, int last, uint16_t* dst, int w) const {
    const char* p = reinterpret_cast<const char*>(src);
    uint16_t* d = dst + w * NI * RPI * DP;
    if (last >= 63) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        __builtin_amdgcn_global_load_lds((gbl_void_t*)(p + off[i]), (lds_void_t*)(d + i * RPI * DP), 16, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int over = max(r0 + i * RPI - last, 0);
        __builtin_amdgcn_global_load_lds((gbl_void_t*)(p + (off[i] - (uint32_t)over * pitch)),
                                         (lds_void_t*)(d + i * RPI * DP), 16, 0, 0);
      }
    }
  }
};

// Byte offsets of a lane's fragment reads within a tile. With the swizzle
// above, the reduction step (or column block) only flips bits of them, and a
// row offset that is a multiple of 16 adds to them: one offset each is kept,
// the others are an exclusive-or away. fresh() hides them from the compiler,
// which otherwise keeps every variant in a register of its own (and spills).
struct LaneOffsets {
  uint32_t row;  // row_frag: row l & 31, chunk h
  uint32_t col;  // col_frag: row 4 h + (s >> 2), columns 16 (g & 1) + 4 (s & 3)
  __device__ __forceinline__ LaneOffsets fresh() const {
    LaneOffsets r = *this;
    asm volatile("" : "+v"(r.row), "+v"(r.col));
    return r;
  }
};
template <int DP>
__device__ __forceinline__ LaneOffsets lane_offsets(int l) {
  const int R = l & 31, g = l >> 4, s = l & 15;
  const int C = 4 * (g >> 1) + (s >> 2), col = 16 * (g & 1) + 4 * (s & 3);
  LaneOffsets o;
  o.row = (uint32_t)(R * DP * 2 + 16 * ((l >> 5) ^ tile_swz<DP>(R)));
  o.col = (uint32_t)(C * DP * 2 + 16 * ((col >> 3) ^ tile_swz<DP>(C)) + 2 * (col & 7));
  return o;
}

// A fragment for rows R0 .. R0 + 31 of a tile (R0 a multiple of 32), reduction
// step ks (16 columns).
template <int DP>
__device__ __forceinline__ bf16x8 row_frag(const uint16_t* t, int R0, int ks, const LaneOffsets& o) {
  return *reinterpret_cast<const bf16x8*>(reinterpret_cast<const char*>(t) + (o.row ^ (32u * ks)) + R0 * DP * 2);
}

// A fragment of the transposed tile: rows are columns 32 db .. + 31 of the
// tile, the reduction runs over its rows R0 .. R0 + 15 (R0 a multiple of 16).
template <int DP>
__device__ __forceinline__ bf16x8 col_frag(const uint16_t* t, int R0, int db, const LaneOffsets& o) {
  const char* p = reinterpret_cast<const char*>(t) + R0 * DP * 2;
  const uint2 a = __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(p + (o.col ^ (64u * db)))));
  const uint2 b = __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(p + (o.col ^ (64u * db + 48u)) + 8 * DP * 2)));
  return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}

// The same for v_mfma_f32_16x16x32_bf16 (A 16 x 32, B 32 x 16): A: lane l
// holds row l & 15, B: column l & 15, each with the 8 reduction places of
// quarter g = l >> 4; D: column l & 15, rows 4 g + 0..3. Two score blocks of 16
// rows make one B fragment, at the rows 4 g + 0..3 and 16 + 4 g + 0..3.
template <int DP>
__device__ __forceinline__ LaneOffsets lane_offsets16(int l) {
  const int R = l & 15, g = l >> 4, C = 4 * g + (R >> 2);
  LaneOffsets o;
  o.row = (uint32_t)(R * DP * 2 + 16 * (g ^ tile_swz<DP>(R)));
  o.col = (uint32_t)(C * DP * 2 + 16 * (((R & 3) >> 1) ^ tile_swz<DP>(C)) + 8 * (R & 1));
  return o;
}
// Rows R0 .. + 15, columns 32 ks .. + 31.
template <int DP>
__device__ __forceinline__ bf16x8 row_frag16(const uint16_t* t, int R0, int ks, const LaneOffsets& o) {
  return *reinterpret_cast<const bf16x8*>(reinterpret_cast<const char*>(t) + (o.row ^ (64u * ks)) + R0 * DP * 2);
}
// Columns 16 db .. + 15 as rows, the tile's rows R0 .. + 31 as the reduction.
template <int DP>
__device__ __forceinline__ bf16x8 col_frag16(const uint16_t* t, int R0, int db, const LaneOffsets& o) {
  const char* p = reinterpret_cast<const char*>(t) + (o.col ^ (32u * db)) + R0 * DP * 2;
  const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)p));
  const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(p + 16 * DP * 2)));
  return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}

// B fragment from 8 values of a score block (registers 8 kb .. + 7).
__device__ __forceinline__ bf16x8 pack_frag(const f32x16& s, int kb) {
  return __builtin_bit_cast(bf16x8, make_uint4(pack_bf16(s[8 * kb], s[8 * kb + 1]), pack_bf16(s[8 * kb + 2], s[8 * kb + 3]),
                                               pack_bf16(s[8 * kb + 4], s[8 * kb + 5]),
                                               pack_bf16(s[8 * kb + 6], s[8 * kb + 7])));
}

// Row of a score block held in register r by half h.
__device__ __forceinline__ constexpr int block_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// B fragment of step ks straight from memory: column (query or key) row
// `p`, 16 ks + 8 h .. + 7; zero where the row or the columns do not exist.
__device__ __forceinline__ bf16x8 global_frag(const uint16_t* p, bool ok, int D, int ks, int l) {
  const int c = 16 * ks + 8 * (l >> 5);
  if (!ok || c >= D) return __builtin_bit_cast(bf16x8, make_uint4(0, 0, 0, 0));
  return *reinterpret_cast<const bf16x8*>(p + c);
}

// Sequence b of a packed batch, its bounds kept inside the arrays whatever
// the starts hold.
struct SeqView {
  int64_t q0, k0;
  int Lq, Lk;
};
__device__ __forceinline__ SeqView seq_view(const AttnArgs& a, int b) {
  SeqView v;
  v.q0 = min(max((int64_t)a.cu_q[b], (int64_t)0), a.Tq);
  v.k0 = min(max((int64_t)a.cu_k[b], (int64_t)0), a.Tk);
  v.Lq = (int)(min(max((int64_t)a.cu_q[b + 1], v.q0), a.Tq) - v.q0);
  v.Lk = (int)(min(max((int64_t)a.cu_k[b + 1], v.k0), a.Tk) - v.k0);
  return v;
}

// Rows first .. last - 1 of head h become zero: share x of n workgroups' work. (Of
// rows that belong to no sequence: an array may be longer than its batch.)
__device__ __forceinline__ void zero_rows(const AttnTensor& t, int h, int64_t first, int64_t last, int D, int x, int n) {
  const int C = D / 8;  // 16-byte chunks of a row
  for (int64_t e = (int64_t)x * blockDim.x + threadIdx.x; e < (last - first) * C; e += (int64_t)n * blockDim.x)
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.p) + (first + e / C) * t.st + h * t.sh + e % C * 8) =
        make_uint4(0, 0, 0, 0);
}

// Workgroup g runs on XCD g % 8. A unit is a sequence's key head; its work is
// `per` items (blocks of rows, times query heads), all of which read the same
// keys and values, so a unit's items run one after another on one XCD and meet
// in its L2. Units are dealt to the XCDs in turn (sequences differ in length);
// fewer than 64 units are cut into `cut` interleaved parts each, so that every
// XCD has work. item = -1: nothing to do.
struct UnitGrid {
  int units, per, cut;
  UnitGrid(int64_t units_, int64_t per_) : units((int)units_), per((int)per_) {
    int64_t c = units_ >= 64 ? 1 : (64 + units_ - 1) / units_;
    if (c > per_) c = per_;
    cut = (int)c;
  }
  int64_t part() const { return (per + cut - 1) / cut; }
  dim3 grid() const { return dim3((unsigned)(8 * (((int64_t)units * cut + 7) / 8) * part())); }
};
// Workgroups along the `blocks` blocks of a unit's head, when there are `all`
// blocks in the launch: with thousands of them a workgroup takes up to `most`
// in turn, which saves it the way from launch to first tile (16 x 512 tokens, 64
// heads of 128, window 256: forward 171 us with two blocks each, 187 with one, 173
// with four; dQ two as well, one costs 10 us more; key blocks 514 us of backward
// with four, 533 with two, 538 with one).
inline int block_groups(int64_t blocks, int64_t all, int64_t most) {
  int64_t m = all / 1024;
  m = m < 1 ? 1 : m > most ? most : m;
  return (int)((blocks + m - 1) / m);
}
// `groups` such groups of a head, or as many as a launch takes of `per` heads
// (or parts) for each of `units` units: a UnitGrid of n per items has at most
// (units + 7) n per + 256 workgroups, its own rounding included. What a group
// does not come to in one turn it does in the next, so fewer cost time only.
inline int fit_groups(int64_t groups, int64_t units, int64_t per, int threads) {
  const int64_t most = (launch_limit(threads) - 256) / ((units + 7) * per);
  return (int)(groups < most ? groups : most < 1 ? 1 : most);
}
struct UnitItem {
  int unit, item;
};
__device__ __forceinline__ UnitItem unit_item(const UnitGrid& g) {
  const int len = (g.per + g.cut - 1) / g.cut;
  const int k = (int)(blockIdx.x >> 3);
  const int part = (int)(blockIdx.x & 7) + 8 * (k / len);
  if (part >= g.units * g.cut) return UnitItem{0, -1};
  const int item = k % len * g.cut + part % g.cut;
  return UnitItem{part / g.cut, item < g.per ? item : -1};
}

// The key tiles of 64 that a workgroup's queries (positions p0 .. p1) can see,
// in the order of the walk: the sinks' tile (tile 0, when it lies in front of
// the window), then the window's tiles; and, for one wave's queries (q0 ..
// q1, none when q1 < q0), which of them hold no or only visible pairs.
struct TileWalk {
  int first;  // 1: the sinks' tile comes first, 0: it does not
  int lo, n;  // first tile of the window, tiles in all
  int jump;   // keys from the sinks' tile to the window
  int any0, any1, all0, all1;  // tiles with any, with only visible pairs by the window
  bool sink;                   // tile 0 holds visible sinks

  __device__ __forceinline__ TileWalk(int p0, int p1, int q0, int q1, int Lk, int window, int sinks) {
    const int hi = min(p1, Lk - 1);
    lo = max(max(p0, 0) - window + 1, 0) >> 6;
    first = sinks > 0 && lo > 0 ? 1 : 0;
    n = hi < 0 ? 0 : first + (hi >> 6) - lo + 1;
    jump = 64 * lo;
    any0 = (max(q0, 0) - window + 1) >> 6;
    any1 = q1 < q0 ? -1 : q1 >> 6;
    all0 = ((max(q1, -1) - window) >> 6) + 1;
    all1 = (max(q0, -1) - 63) >> 6;
    sink = sinks > 0 && q1 >= q0 && q1 >= 0;
  }
  __device__ __forceinline__ int tile(int i) const { return first && i == 0 ? 0 : lo + i - first; }
  __device__ __forceinline__ bool hidden(int t) const { return (t < any0 || t > any1) && !(t == 0 && sink); }
  __device__ __forceinline__ bool edge(int t) const { return t < all0 || t > all1; }
};
// Address of the walk's next tile.
struct TileSource {
  const uint16_t* p;
  int64_t step, jump;
  __device__ __forceinline__ TileSource(const uint16_t* base, int64_t pitch, const TileWalk& w)
      : p(base + (w.first ? 0 : w.jump * pitch)), step(64 * pitch), jump(w.jump * pitch) {}
  __device__ __forceinline__ void next(int i, const TileWalk& w) { p += i + 1 == w.first ? jump : step; }
};

// Waits until at most n of this wave's memory instructions are in flight
// (their order of issue is the order of completion that vmcnt counts), and
// for its LDS reads.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
}
// Tile i of n is about to be read, PER memory instructions bring a tile, tiles
// up to i + AHEAD have been asked for.
template <int PER, int AHEAD>
__device__ __forceinline__ void wait_tile(int i, int n) {
  static_assert(AHEAD >= 0 && AHEAD <= 2, "tiles in flight");
  if (AHEAD >= 2 && i + 2 < n) wait_vm<2 * PER>();
  else if (AHEAD >= 1 && i + 1 < n) wait_vm<PER>();
  else wait_vm<0>();
}

// Hides the pairs of a score block that are not seen: columns are queries (one
// per lane, position pos), rows the keys j0 + block_row(r, h). All the
// differences are small: the tile holds a key that some query of the
// workgroup sees.
__device__ __forceinline__ void hide_keys(f32x16& s, float with, int j0, int pos, int window, int sinks, int l) {
  const int rel = pos - j0 - 4 * (l >> 5), low = rel - window, first = sinks - j0 - 4 * (l >> 5);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int i = block_row(r, 0);
    const bool see = (i <= rel) & ((i > low) | (i < first));
    s[r] = see ? s[r] : with;
  }
}

}  // namespace qlora
