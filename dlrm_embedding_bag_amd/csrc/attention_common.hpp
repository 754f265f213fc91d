// attention_common.hpp -- internal helpers of the attention kernels: packed
// sequences and their tiles, tiles of rows in LDS, and matrix products of 32 x 32
// outputs over 16 contracted elements, in bfloat16 or float32.
#pragma once

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The product of 32 x 32 outputs, out[m][n] += sum over 16 k of a[m][k] b[n][k].
// A lane holds eight k of one row of a (row lane % 32) and of one of b, those
// with k / 8 % 2 == lane / 32 or any other order that a and b share; of the
// outputs it holds column lane % 32 and rows row_of(i, lane / 32).
// float32 goes by eight products over two k, each lane's own element of each.
template <typename T>
struct Operand;
template <>
struct Operand<BF16> {
  u32x4_t v;
};
template <>
struct Operand<F32> {
  f32x4_t v[2];
};

__device__ __forceinline__ constexpr int row_of(int i, int half) {
  return (i >> 2) * 8 + half * 4 + (i & 3);
}

__device__ __forceinline__ f32x16_t multiply(const Operand<BF16> &a, const Operand<BF16> &b,
                                             f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a.v),
                                                 __builtin_bit_cast(bf16x8_t, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t multiply(const Operand<F32> &a, const Operand<F32> &b,
                                             f32x16_t c) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[e >> 2][e & 3], b.v[e >> 2][e & 3], c, 0, 0, 0);
  return c;
}

// Outputs 8m .. 8m + 7 of a lane as the operand of a product over the 16 rows
// that they and the other half's hold: slot e of half h stands for row
// row_of(8m + e, h).
template <typename T>
__device__ __forceinline__ Operand<T> operand_of(const f32x16_t &c, int m) {
  Operand<T> o;
  if constexpr (sizeof(typename T::S) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o.v[e >> 2][e & 3] = c[8 * m + e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) o.v[e] = pack_bf16(c[8 * m + 2 * e], c[8 * m + 2 * e + 1]);
  }
  return o;
}

template <typename T>
__device__ __forceinline__ Operand<T> zero_operand() {
  Operand<T> o{};
  return o;
}

// Eight elements from c on of a row of memory, zeros where there is no row or
// c lies beyond its end (rows hold a multiple of eight).
template <typename T>
__device__ __forceinline__ Operand<T> load_operand(const typename T::S *row, int c, int dim,
                                                   bool there) {
  Operand<T> o = zero_operand<T>();
  if (there && c < dim) {
    if constexpr (sizeof(typename T::S) == 4) {
      o.v[0] = *reinterpret_cast<const f32x4_t *>(row + c);
      o.v[1] = *reinterpret_cast<const f32x4_t *>(row + c + 4);
    } else {
      o.v = *reinterpret_cast<const u32x4_t *>(row + c);
    }
  }
  return o;
}

// ------------------------------------------------------------ tiles in LDS --
// ROWS rows of DP elements as chunks of 16 bytes.  Chunk c of row r lies at
// place c ^ (2 (r & 3) + (r >> 2 & 1)): eight rows read at one chunk start on
// different banks, and so do two chunks each of four rows, which is what a
// transposed read takes.
template <typename T, int ROWS, int DP>
struct LdsTile {
  using S = typename T::S;
  static constexpr int E = 16 / sizeof(S);                 // elements of a chunk
  static constexpr int C = DP == 96 ? 128 / E : DP / E;    // places of a row, a power of two
  static constexpr int MASK = C < 8 ? C - 1 : 7;
  static constexpr int SIZE = ROWS * C;                    // chunks

  __device__ __forceinline__ static int key(int row) {
    return ((row & 3) << 1 | (row >> 2 & 1)) & MASK;
  }
};

// `bytes` of memory from `base` on, behind which loads read zeros.  (These two
// are no templates: the host's pass drops kernels whose templates call such
// builtins twice.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 4 << 15);
}
// 16 or 4 bytes a lane, from memory to LDS: lane l's to lds[l].
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t from,
                                            u32x4_t *lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds, 16, from, 0, 0, 0);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t from, float *lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds, 4, from, 0, 0, 0);
}

// What a thread asks for when a tile is filled: where its chunks lie in memory,
// relative to the tile's first row.
template <typename T, int ROWS, int DP, int WAVES>
struct TileLoad {
  using L = LdsTile<T, ROWS, DP>;
  static constexpr int LOADS = L::SIZE / (WAVES * kWave);
  static_assert(L::SIZE % (WAVES * kWave) == 0);
  static constexpr uint32_t kNowhere = 0x80000000u;  // beyond any tile: reads as zeros
  uint32_t from[LOADS];

  __device__ __forceinline__ TileLoad(int wave, int lane, int64_t row_stride, int dim) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int at = (i * WAVES + wave) * kWave + lane;
      const int r = at / L::C, c = ((at % L::C) ^ L::key(r)) * L::E;
      from[i] = c < dim ? (uint32_t)((r * row_stride + c) * (int64_t)sizeof(typename T::S))
                        : kNowhere;
    }
  }
  // Rows `base` on, of which `rows` are there (the others become zeros); the
  // loads are on their way when this returns.
  __device__ __forceinline__ void fill(u32x4_t *lds, const typename T::S *base, int64_t rows,
                                       int64_t row_stride, int dim, int wave) const {
    const int n = rows < ROWS ? (int)rows : ROWS;
    const uint32_t bytes =
        n > 0 ? (uint32_t)(((n - 1) * row_stride + dim) * (int64_t)sizeof(typename T::S)) : 0;
    const auto b = buffer_of(base, bytes);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_to_lds(b, from[i], lds + (i * WAVES + wave) * kWave);
  }
};

// Row r0 + lane % 32 of a tile, elements 16 step + 8 (lane / 32) on: the operand
// of a product over the row's elements.
template <typename T, int ROWS, int DP>
__device__ __forceinline__ Operand<T> read_rows(const u32x4_t *lds, int r0, int step, int lane) {
  using L = LdsTile<T, ROWS, DP>;
  const int r = lane & 31, h = lane >> 5;
  const u32x4_t *row = lds + (r0 + r) * L::C;
  Operand<T> o;
  if constexpr (L::E == 8) {
    o.v = row[(step * 2 + h) ^ L::key(r)];
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      o.v[e] = __builtin_bit_cast(f32x4_t, row[(step * 4 + h * 2 + e) ^ L::key(r)]);
  }
  return o;
}

// Column d0 + lane % 32 of a tile, its rows r0 + row_of(e, lane / 32) in slots e
// of 0..7: the operand of a product over 16 rows (r0 a multiple of 16).  For
// bfloat16 by the transposing read: of 16 lanes each gives the place of four
// elements, and gets one element of each of the four rows they span.
template <typename T, int ROWS, int DP>
__device__ __forceinline__ Operand<T> read_columns(const u32x4_t *lds, int r0, int d0, int lane) {
  using L = LdsTile<T, ROWS, DP>;
  Operand<T> o;
  const int h = lane >> 5;
  if constexpr (L::E == 8) {
    typedef __attribute__((address_space(3))) i16x4_t *Quad;
    const int i = lane & 15;
    const int c = d0 / 8 + (lane >> 4 & 1) * 2 + (i >> 1 & 1);
    const int t = h * 4 + (i >> 2);
    const char *at = (const char *)(lds + (r0 + t) * L::C + (c ^ L::key(t))) + (i & 1) * 8;
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Quad)at);
    const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Quad)(at + 8 * L::C * 16));
    const auto a = __builtin_bit_cast(u32x2_u, lo), b = __builtin_bit_cast(u32x2_u, hi);
    o.v = u32x4_t{a[0], a[1], b[0], b[1]};
  } else {
    const int d = d0 + (lane & 31);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = row_of(e, h);
      o.v[e >> 2][e & 3] =
          reinterpret_cast<const float *>(lds + (r0 + t) * L::C + ((d >> 2) ^ L::key(t)))[d & 3];
    }
  }
  return o;
}

// Loads to LDS and LDS accesses of this wave are done, and everyone's.
__device__ __forceinline__ void landed() {
  __builtin_amdgcn_s_waitcnt(0x0070);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// -------------------------------------------------------- packed sequences --
// Sequence b of a packed batch holds rows offsets[b] .. offsets[b + 1] - 1.
// With the rows before the first and behind the last these are batch + 2
// segments, and tiles of `rows` rows are numbered so that segment s begins at
// tile start(s) / rows + s: that leaves each segment as many tiles as it needs
// (a few too many), grows with s, and takes no table.  A tile is found by a
// search for its segment, 64 at a time.
struct Tile {
  int64_t sequence;     // -1: outside all sequences
  int64_t first, last;  // rows of the segment
  int64_t row;          // first row of the tile; none where it is >= last
};

// Where segment s begins, and the last one ends; offsets that a bad array holds
// are moved into the tensor.
__device__ __forceinline__ int64_t segment_start(const int32_t *offsets, int64_t batch,
                                                 int64_t total, int64_t s) {
  if (s <= 0) return 0;
  if (s > batch + 1) return total;
  const int64_t o = offsets[s - 1];
  return o < 0 ? 0 : o > total ? total : o;
}

__host__ __device__ inline int64_t tile_count(int64_t total, int64_t batch, int rows) {
  return total / rows + batch + 2;
}

// Every lane of the wave takes part; the result is the same in all.
__device__ __forceinline__ Tile find_tile(const int32_t *offsets, int64_t batch, int64_t total,
                                          int64_t tile, int rows) {
  const int lane = threadIdx.x % kWave;
  int64_t lo = 0, n = batch + 2;  // the segment is one of [lo, lo + n)
  while (n > 1) {
    const int64_t step = (n + kWave - 1) / kWave;
    const int64_t s = lo + lane * step;
    bool before = false;
    if (s < lo + n) before = segment_start(offsets, batch, total, s) / rows + s <= tile;
    const uint64_t mask = __ballot(before);
    const int64_t last = mask ? 63 - __clzll(mask) : 0;
    const int64_t end = lo + n;
    lo += last * step;
    n = end - lo < step ? end - lo : step;
  }
  lo = (int64_t)__builtin_amdgcn_readfirstlane((uint32_t)lo) |
       (int64_t)__builtin_amdgcn_readfirstlane((uint32_t)(lo >> 32)) << 32;
  Tile t;
  t.sequence = lo >= 1 && lo <= batch ? lo - 1 : -1;
  t.first = segment_start(offsets, batch, total, lo);
  t.last = segment_start(offsets, batch, total, lo + 1);
  const int64_t k = tile - (t.first / rows + lo);
  t.row = k < 0 ? t.last : t.first + k * rows;
  return t;
}

// The keys of a tile's sequence.
struct KeyRange {
  int64_t first, count;
};
__device__ __forceinline__ KeyRange keys_of(const int32_t *offsets, const int32_t *kv_offsets,
                                            int64_t batch, int64_t kv_tokens, const Tile &t) {
  if (!kv_offsets) return {t.first, t.last - t.first};
  const int64_t first = segment_start(kv_offsets, batch, kv_tokens, t.sequence + 1);
  const int64_t last = segment_start(kv_offsets, batch, kv_tokens, t.sequence + 2);
  return {first, last > first ? last - first : 0};
}

// How many of them, from the first on, are seen: all, or with `causal` by the
// last row all and by each row before it one less.
struct SeenKeys {
  int64_t mine;      // by this lane's row
  int64_t wave_all;  // by every row of the wave's 32
  int64_t wave_any;  // by any of them
  int64_t tile_any;  // by any row of the workgroup's tile
  __device__ __forceinline__ SeenKeys(int causal, int64_t keys, int64_t last, int64_t tile_row,
                                      int tile_rows, int wave, int64_t row, bool there) {
    auto by = [&](int64_t r) {
      const int64_t n = causal ? keys - (last - 1 - r) : keys;
      return n < 0 ? 0 : n;
    };
    auto end = [&](int64_t r) { return r < last - 1 ? r : last - 1; };
    const int64_t first = tile_row + wave * 32;
    mine = there ? by(row) : 0;
    wave_all = first + 31 < last ? by(first) : 0;
    wave_any = first < last ? by(end(first + 31)) : 0;
    tile_any = by(end(tile_row + tile_rows - 1));
  }
};

// Workgroups for that many items; each takes those a grid apart.
inline uint32_t grid_of(int64_t items) {
  return (uint32_t)(items < (1 << 22) ? items : 1 << 22);
}

}  // namespace dlrm
