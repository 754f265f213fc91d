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
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

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

// ------------------------------------------------------------ tiles in LDS --
// ROWS rows of DP elements as chunks of 16 bytes, C places a row.  LDS serves 256
// bytes at once: 16 lanes of a row's read (16 rows, one chunk), 32 of a transposed
// one (4 neighbouring rows, 4 neighbouring chunks), 64 of single floats (rows t and
// t + 4, 8 neighbouring chunks).  So that none of these meet on a bank, chunk c of
// row r lies at place c ^ key(r), where the places of 16 rows differ and
//   bfloat16  four neighbouring rows differ in the key's upper two bits,
//   float32   rows t and t + 4 in its uppermost.
// (Of 64 keys and values in bfloat16 at dim 128 a read takes 4 cycles, or 2 if
// transposed; with a three-bit key for eight rows 8 and 4.)
template <typename T, int ROWS, int DP>
struct LdsTile {
  using S = typename T::S;
  static constexpr int E = 16 / sizeof(S);                 // elements of a chunk
  static constexpr int C = DP == 96 ? 128 / E : DP / E;    // places of a row, a power of two
  static constexpr int SIZE = ROWS * C;                    // chunks
  static constexpr int BITS = C >= 16 ? 15 : C - 1;        // of a key

  // of a row in 0 .. 15; keys repeat every 16 rows
  __device__ __forceinline__ static int key(int row) {
    if constexpr (E == 8)
      return C >= 16  ? (row & 3) << 2 | (row >> 2 & 3)
             : C == 8 ? (row & 2) << 1 | (row >> 2 & 3)     // two rows are 256 bytes
                      : row >> 2 & 3;                       // four rows are
    else
      return C >= 16 ? (row & 4) << 1 | (row & 3) << 1 | (row >> 3 & 1) : row >> 1 & 7;
  }
};

// Tiles are passed by their addresses in LDS.
typedef __attribute__((address_space(3))) u32x4_t *LdsChunks;
typedef __attribute__((address_space(3))) float *LdsFloats;
typedef const __attribute__((address_space(3))) char *LdsBytes;

// `bytes` of memory from `base` on, behind which loads read zeros.  (These are no
// templates: the host's pass drops kernels whose templates call such builtins
// twice.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 4 << 15);
}
constexpr uint32_t kNowhere = 0x80000000u;   // an offset beyond any such buffer
// 16 bytes from there to registers, and 16 or 8 back; stores beyond it do nothing.
__device__ __forceinline__ u32x4_t load_from(__amdgpu_buffer_rsrc_t b, uint32_t from) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(b, from, 0, 0));
}
__device__ __forceinline__ void store_to(__amdgpu_buffer_rsrc_t b, uint32_t to, u32x4_t v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, b, to, 0, 0);
}
__device__ __forceinline__ void store_to(__amdgpu_buffer_rsrc_t b, uint32_t to, u32x2_t v) {
  __builtin_amdgcn_raw_buffer_store_b64(v, b, to, 0, 0);
}
// 16 or 4 bytes a lane, from memory to LDS: lane l's to lds[l].
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t from,
                                            LdsChunks lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds, 16, from, 0, 0, 0);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t from, LdsFloats lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds, 4, from, 0, 0, 0);
}

// A value that every lane of the wave holds alike, for the scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// Fills tiles one after another with the rows of a tensor: a wave's loads keep
// their lanes' offsets, and only the buffer moves on.  Behind the last row a tile
// holds zeros, or where rows repeat (a stride below their length) one of them.
template <typename T, int ROWS, int DP, int WAVES>
struct TileLoad {
  using S = typename T::S;
  using L = LdsTile<T, ROWS, DP>;
  static constexpr int LOADS = L::SIZE / (WAVES * kWave);
  static_assert(L::SIZE % (WAVES * kWave) == 0 && WAVES * kWave % L::C == 0);
  uint32_t from[LOADS];
  const S *next;        // the first row of the next tile
  int left;             // rows from there on
  int64_t stride;       // elements of a row

  __device__ __forceinline__ TileLoad(int wave, int lane, int64_t row_stride, int dim)
      : stride(row_stride) {
    // row r0 + i STEP of load i; the key of a sum of disjoint bits is the exclusive
    // or of their keys
    constexpr int STEP = WAVES * kWave / L::C;
    const int at = wave * kWave + lane, r0 = at / L::C;
    const uint32_t place = at % L::C ^ L::key(r0 & 15);
    const uint32_t row = (uint32_t)row_stride * (uint32_t)sizeof(S), at0 = r0 * row;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const uint32_t c = place ^ L::key(i * STEP & 15);
      from[i] = c * L::E < (uint32_t)dim ? c * 16 + (at0 + i * STEP * row) : kNowhere;
    }
  }
  __device__ __forceinline__ void start(const S *base, int rows) {
    next = base;
    left = rows;
  }
  // The loads are on their way when this returns.
  __device__ __forceinline__ void fill(LdsChunks lds, int dim, int wave) {
    const uint32_t rows = left < ROWS ? left : ROWS;
    const auto b = buffer_of(next, ((rows - 1) * (uint32_t)stride + dim) * (uint32_t)sizeof(S));
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_to_lds(b, from[i], lds + (i * WAVES + wave) * kWave);
    skip(ROWS);
  }
  __device__ __forceinline__ void skip(int rows) {
    next += rows * stride;
    left -= rows;
  }
};

// Where two groups of WAVES waves that share their rows or keys meet at the end: the
// four buffers of their tiles (SIZE chunks each for a group) take 16 sums of each lane
// at a time.
template <int WAVES, int SIZE>
struct Meeting {
  static constexpr int EACH = 2 * SIZE * 16 / (WAVES * kWave * 64);   // of a buffer
  static_assert(EACH >= 1);
  LdsChunks buffers[4];
  int at;
  __device__ __forceinline__ LdsChunks place(int i, int e) const {
    return buffers[i / EACH] + (i % EACH * 4 + e) * WAVES * kWave + at;
  }
  __device__ __forceinline__ void put(int i, const f32x16_t &a) const {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *place(i, e) = u32x4_t{__float_as_uint(a[4 * e]), __float_as_uint(a[4 * e + 1]),
                             __float_as_uint(a[4 * e + 2]), __float_as_uint(a[4 * e + 3])};
  }
  __device__ __forceinline__ void add(int i, f32x16_t &a, float scale = 1.0f) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const u32x4_t w = *place(i, e);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[4 * e + j] = __builtin_fmaf(__uint_as_float(w[j]), scale, a[4 * e + j]);
    }
  }
};

// A lane's row of a tile of rows in memory: rows from `base` on, of which `left`
// are there.  What lies behind them or behind a row's end reads as zeros and is not
// stored.
template <typename T>
struct MemoryRow {
  using S = typename T::S;
  __amdgpu_buffer_rsrc_t buffer;
  uint32_t row;   // offset of the lane's
  int dim;
  __device__ __forceinline__ MemoryRow(const void *base, int64_t stride, int left, int dim_, int r)
      : buffer(buffer_of(base, ((uint32_t)(left < 128 ? left - 1 : 127) * (uint32_t)stride + dim_) *
                                   (uint32_t)sizeof(S))),
        row(r < left ? (uint32_t)r * (uint32_t)stride * (uint32_t)sizeof(S) : kNowhere), dim(dim_) {}
  // Elements 8 c on.
  __device__ __forceinline__ Operand<T> load(int c) const {
    const uint32_t from = c < dim ? row + c * (uint32_t)sizeof(S) : kNowhere;
    Operand<T> o;
    if constexpr (sizeof(S) == 4) {
      o.v[0] = __builtin_bit_cast(f32x4_t, load_from(buffer, from));
      o.v[1] = __builtin_bit_cast(f32x4_t, load_from(buffer, from + 16));
    } else {
      o.v = load_from(buffer, from);
    }
    return o;
  }
  // A lane's half of a row: what its columns of products hold, times `scale`.
  template <int DT>
  __device__ __forceinline__ void store(const f32x16_t (&o)[DT], float scale, int half) const {
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int c = d * 32 + row_of(i, 0);   // (and four more for the other half: rows
        const uint32_t to =                    // hold a multiple of eight)
            c < dim ? row + (c + half * 4) * (uint32_t)sizeof(S) : kNowhere;
        const float w[4] = {o[d][i] * scale, o[d][i + 1] * scale, o[d][i + 2] * scale,
                            o[d][i + 3] * scale};
        if constexpr (sizeof(S) == 4)
          store_to(buffer, to, u32x4_t{__float_as_uint(w[0]), __float_as_uint(w[1]),
                                       __float_as_uint(w[2]), __float_as_uint(w[3])});
        else
          store_to(buffer, to, u32x2_t{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3])});
      }
  }
};

// What a lane reads of tiles: the place of its first chunk, or element.  Others
// differ from it by an exclusive or with a constant, which takes a column and a
// row's key along, and by whole rows.  here() keeps those exclusive ors where they
// are used, for kernels that have no registers to hold them in.
template <typename V>
__device__ __forceinline__ V lds_at(LdsBytes lds, uint32_t place) {
  return *(const __attribute__((address_space(3))) V *)(lds + place);
}

// Row r0 + lane % 32 of a tile, elements 16 step + 8 (lane / 32) on: the operand
// of a product over the row's elements.
template <typename T, int ROWS, int DP>
struct ReadRows {
  using L = LdsTile<T, ROWS, DP>;
  uint32_t place;
  __device__ __forceinline__ explicit ReadRows(int lane) {
    const int r = lane & 31, c = (lane >> 5) * (8 / L::E);
    place = (uint32_t)(r * L::C + (c ^ L::key(r & 15))) * 16;
  }
  __device__ __forceinline__ void here() { asm volatile("" : "+v"(place)); }
  __device__ __forceinline__ Operand<T> read(LdsChunks lds, int r0, int step) const {
    Operand<T> o;
    if constexpr (L::E == 8) {
      o.v = lds_at<u32x4_t>((LdsBytes)lds, (place ^ step * 32) + r0 * L::C * 16);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)   // 16 chunks are four steps
        o.v[e] = lds_at<f32x4_t>((LdsBytes)lds, (place ^ ((step & 3) * 4 + e) * 16) +
                                          (r0 * L::C + step / 4 * 16) * 16);
    }
    return o;
  }
};

// Column 32 d + lane % 32 of a tile, its rows r0 + row_of(e, lane / 32) in slots e
// of 0..7: the operand of a product over 16 rows (r0 a multiple of 16).  For
// bfloat16 by the transposing read: of 16 lanes each gives the place of four
// elements, and gets one element of each of the four rows they span.
template <typename T, int ROWS, int DP>
struct ReadColumns {
  using L = LdsTile<T, ROWS, DP>;
  uint32_t place;
  __device__ __forceinline__ explicit ReadColumns(int lane) {
    const int h = lane >> 5;
    if constexpr (L::E == 8) {
      const int q = lane & 15, t = h * 4 + (q >> 2), c = (lane >> 4 & 1) * 2 + (q >> 1 & 1);
      place = (uint32_t)(t * L::C + (c ^ L::key(t))) * 16 + (q & 1) * 8;
    } else {
      const int t = h * 4, c = (lane & 31) >> 2;
      place = (uint32_t)(t * L::C + (c ^ L::key(t))) * 16 + (lane & 3) * 4;
    }
  }
  __device__ __forceinline__ void here() { asm volatile("" : "+v"(place)); }
  __device__ __forceinline__ Operand<T> read(LdsChunks lds, int r0, int d) const {
    Operand<T> o;
    if constexpr (L::E == 8) {
      typedef __attribute__((address_space(3))) i16x4_t *Quad;
      const LdsBytes at = (LdsBytes)lds + r0 * L::C * 16;
      const uint32_t by_key = (L::key(8) ^ d * 4) * 16;
      const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Quad)(at + (place ^ d * 64)));
      const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (Quad)(at + ((place ^ by_key) + 8 * L::C * 16)));
      const auto a = __builtin_bit_cast(u32x2_u, lo), b = __builtin_bit_cast(u32x2_u, hi);
      o.v = u32x4_t{a[0], a[1], b[0], b[1]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = row_of(e, 0);                   // (rows t and t + 4 differ by a bit
        const uint32_t by_key = (L::key(t) ^ (d & 1) * 8) * 16;  // that the place has)
        o.v[e >> 2][e & 3] = lds_at<float>(
            (LdsBytes)lds, (place ^ by_key) + ((r0 + t) * L::C + (L::C > 8 ? d / 2 * 16 : 0)) * 16);
      }
    }
    return o;
  }
};

// Waves of a SIMD that a kernel leaves registers for: two cover each other's waits,
// but float32 rows of more than 64 would spill (gradient of 2 x 2000 rows, 8 heads of
// 128: one wave 1361 us, two 1892).
template <typename T, int DP>
constexpr int waves_a_simd = sizeof(typename T::S) == 4 && DP > 64 ? 1 : 2;

// Loads to LDS and LDS accesses of this wave are done, and everyone's.
__device__ __forceinline__ void landed() {
  __builtin_amdgcn_s_waitcnt(0x0070);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// N products in order, whose operands `read(i)` brings from LDS: each read stands
// AHEAD products before its own, so that none waits for LDS.  PINNED: in just this
// order (where nothing else is to do, the compiler saves registers and has each
// product wait for its own read).
template <typename T, int N, int AHEAD, bool PINNED, typename Read, typename Use>
__device__ __forceinline__ void in_order(Read &&read, Use &&use) {
  constexpr int A = AHEAD < N ? AHEAD : N;
  Operand<T> a[A];
#pragma unroll
  for (int i = 0; i < A; ++i) a[i] = read(i);
  if (PINNED) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Operand<T> now = a[i % A];
    if (i + A < N) a[i % A] = read(i + A);
    use(i, now);
    if (PINNED) __builtin_amdgcn_sched_barrier(0);
  }
}

// -------------------------------------------------------- packed sequences --
// Sequence b of a packed batch holds rows offsets[b] .. offsets[b + 1] - 1.
// With the rows before the first and behind the last these are batch + 2
// segments, and tiles of `rows` rows are numbered so that segment s begins at
// tile start(s) / rows + s: that leaves each segment as many tiles as it needs
// (a few too many), grows with s, and takes no table.  A tile is found by a
// search for its segment, 64 at a time.
struct Tile {
  int sequence;     // -1: outside all sequences
  int first, row;   // rows: the segment's first, the tile's first
  int left;         // rows from there to the segment's end; none where it is <= 0
};

// Where segment s begins, and the last one ends; offsets that a bad array holds
// are moved into the tensor.
__device__ __forceinline__ int segment_start(const int32_t *offsets, uint32_t batch, int total,
                                             uint32_t s) {
  if (s == 0) return 0;
  if (s > batch + 1) return total;
  const int o = offsets[s - 1];
  return o < 0 ? 0 : o > total ? total : o;
}

__host__ __device__ inline int64_t tile_count(int64_t total, int64_t batch, int rows) {
  return total / rows + batch + 2;   // (below 2^32)
}

// Every lane of the wave takes part; the result is the same in all.
__device__ __forceinline__ Tile find_tile(const int32_t *offsets, uint32_t batch, int total,
                                          uint32_t tile, uint32_t rows) {
  const uint32_t lane = threadIdx.x % kWave;
  uint32_t lo = 0, n = batch + 2;  // the segment is one of [lo, lo + n)
  while (n > 1) {
    const uint32_t step = (n - 1) / kWave + 1;
    const uint32_t s = lo + lane * step;   // (below 2^32: n is below 2^31 + 2)
    bool before = false;
    if (lane * step < n)
      before = (uint32_t)segment_start(offsets, batch, total, s) / rows + s <= tile;
    const uint64_t mask = __ballot(before);
    const uint32_t last = mask ? 63 - __clzll(mask) : 0;
    lo = (uint32_t)uniform((int)(lo + last * step));
    n = n - last * step < step ? n - last * step : step;
    n = (uint32_t)uniform((int)n);
  }
  const int first = uniform(segment_start(offsets, batch, total, lo));
  const int last = uniform(segment_start(offsets, batch, total, lo + 1));
  const uint32_t start = (uint32_t)first / rows + lo;
  const uint64_t row = (uint64_t)first + (uint64_t)(tile - start) * rows;
  Tile t;
  t.sequence = lo >= 1 && lo <= batch ? (int)lo - 1 : -1;
  t.first = first;
  const bool there = tile >= start && row < (uint64_t)(last > 0 ? last : 0);
  t.left = there ? (int)(last - (int64_t)row) : 0;
  t.row = there ? (int)row : last;
  return t;
}

// The rows of sequence b in the other tensor.
struct Range {
  int first, count;
};
__device__ __forceinline__ Range rows_of(const int32_t *offsets, uint32_t batch, int total, int b) {
  const int first = uniform(segment_start(offsets, batch, total, (uint32_t)b + 1));
  const int last = uniform(segment_start(offsets, batch, total, (uint32_t)b + 2));
  return {first, last > first ? last - first : 0};
}

// How many keys, from the first on, are seen: all, or with `causal` by the last
// row all and by each row before it one less.  Rows count from the tile's first,
// of which the tile has `tile_rows`, this wave `wave_rows`.
struct SeenKeys {
  int causal, keys, left;
  int wave_all;  // by every row of the wave (that is there)
  int wave_any;  // by any of them
  int tile_all;  // by every row of the workgroup's tile
  int tile_any;  // by any of them
  __device__ __forceinline__ SeenKeys(int causal_, int keys_, int rows_left, int tile_rows,
                                      int wave, int wave_rows)
      : causal(causal_), keys(keys_), left(rows_left) {
    const int first = wave * wave_rows;
    wave_all = by(first);
    wave_any = first < left ? by(end(first + wave_rows - 1)) : 0;
    tile_all = by(0);
    tile_any = by(end(tile_rows - 1));
  }
  __device__ __forceinline__ int end(int r) const { return r < left - 1 ? r : left - 1; }
  __device__ __forceinline__ int by(int r) const {   // 0 for a row that is not there
    const int n = causal ? keys - (left - 1 - r) : keys;
    return n < 0 || r >= left ? 0 : n;
  }
};

// Item `i` of tiles * heads.  The last tiles come first: with `causal` they see
// the most keys, and work that ends early should be short.  Workgroups go to the
// eight dies in turn, so a die gets heads that lie together, whose key heads then
// share its cache (both together: four prompts of up to 6500 rows 955 us for 1019).
struct Item {
  uint32_t tile;
  int head;
};
__device__ __forceinline__ Item item_of(int64_t i, int64_t tiles, int heads) {
  const uint64_t n = (uint64_t)i;
  int64_t t;
  uint32_t r;
  if (n >> 32) {
    t = (int64_t)(n / (uint32_t)heads);
    r = (uint32_t)(n - (uint64_t)t * heads);
  } else {
    t = (uint32_t)n / (uint32_t)heads;
    r = (uint32_t)n - (uint32_t)t * (uint32_t)heads;
  }
  if (heads % 8 == 0) r = r % 8 * (heads / 8) + r / 8;
  return {(uint32_t)(tiles - 1 - t), (int)r};
}

// Calls of few sequences and not many workgroups: their tiles go out by the keys that
// they see, most first, and where a CU holds PAIRS every second 256 of them in reverse,
// so that one of its two is long where the other is short.  (Seven pieces after 777
// keys, 468 workgroups: 45 us for 50; three sequences of up to 2500, 12 heads of 128, in
// float32 637 for 794; one of 1466 keys in 80 pays 2.5 us for the search.)
__device__ __forceinline__ bool in_order_of_work(int64_t items, int64_t batch, int64_t kv_tokens) {
  return items > 256 && items <= 1024 && batch <= 16 && kv_tokens < 1 << 30;
}
template <bool PAIRS>
__device__ __forceinline__ int64_t pair_up(int64_t item, int64_t items) {
  const int i = (int)item, n = (int)items, at = i & 255, block = i - at;
  return PAIRS && block & 256 ? block + (n - block < 256 ? n - block : 256) - 1 - at : i;
}
// The tile of ROWS rows that is number `rank` in that order; behind them come those
// outside all sequences.  The least number of keys that it may see is found by
// counting, for a number in each lane.
template <int ROWS>
__device__ __forceinline__ Tile tile_of_rank(const int32_t *offsets, const int32_t *kv_offsets,
                                             uint32_t batch, int total, int kv_total, int causal,
                                             int rank) {
  const uint32_t lane = threadIdx.x % kWave;
  int first = 0, rows = 0, keys = 0;   // of the lane's sequence
  if (lane < batch) {
    first = segment_start(offsets, batch, total, lane + 1);
    const int last = segment_start(offsets, batch, total, lane + 2);
    rows = last > first ? last - first : 0;
    keys = rows;
    if (kv_offsets) {
      keys = segment_start(kv_offsets, batch, kv_total, lane + 2) -
             segment_start(kv_offsets, batch, kv_total, lane + 1);
      keys = keys > 0 ? keys : 0;
    }
  }
  // tiles of a sequence that see `least` keys or more: its last ones
  auto seeing = [&](int rows, int keys, int least) __attribute__((always_inline)) {
    const int end = causal && least > 0 ? rows - keys + least : 0;   // rows to a tile's end
    const int none = end > 0 ? (end - 1) / ROWS : 0;
    return least > keys ? 0 : (rows + ROWS - 1) / ROWS - none;
  };
  auto count = [&](int least) __attribute__((always_inline)) {
    int n = 0;
    for (uint32_t b = 0; b < batch; ++b)
      n += seeing(__builtin_amdgcn_readlane(rows, b), __builtin_amdgcn_readlane(keys, b), least);
    return n;
  };
  Tile t;
  const int all = uniform(count(0));
  if (rank >= all) {
    rank -= all;
    const int before = uniform(segment_start(offsets, batch, total, 1));
    const int behind = uniform(segment_start(offsets, batch, total, batch + 1));
    const int n = (before + ROWS - 1) / ROWS;
    t.sequence = -1;
    t.first = rank < n ? 0 : behind;
    const int64_t row = t.first + (int64_t)(rank < n ? rank : rank - n) * ROWS;
    const int last = rank < n ? before : total;
    t.row = row < last ? (int)row : last;
    t.left = last - t.row;
    return t;
  }
  int most = 0, span = 1 << 30;   // it sees most .. most + span - 1
  while (span > 1) {
    const int step = __any(keys - most >= span / 64) ? span / 64 : span / 4096;
    const int each = step > 0 ? step : 1;
    const uint64_t mask = __ballot(count(most + (int)lane * each) > rank);
    most += (63 - __builtin_clzll(mask | 1)) * each;
    span = each;
  }
  rank -= uniform(count(most + 1));
  const int at_most = seeing(rows, keys, most), mine = at_most - seeing(rows, keys, most + 1);
  int upto = mine;
#pragma unroll
  for (int x = 1; x < 16; x *= 2) {
    const int other = __shfl_up(upto, x);
    upto += (int)lane >= x ? other : 0;
  }
  const uint64_t mask = __ballot(lane < batch && upto > rank);
  const int b = mask ? __builtin_ctzll(mask) : 0;
  const int n = (rows + ROWS - 1) / ROWS, tile = n - at_most + rank - (upto - mine);
  t.sequence = b;
  t.first = __builtin_amdgcn_readlane(first, b);
  t.row = t.first + __builtin_amdgcn_readlane(tile, b) * ROWS;
  t.left = t.first + __builtin_amdgcn_readlane(rows, b) - t.row;
  return t;
}

// A scalar whose uses stay within the loop over items: what follows from it would
// else be made before the loop and kept, beyond the registers that there are.
__device__ __forceinline__ int in_loop(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

// What the gradient's second kernel needs of a row, head by head in planes of
// `tokens`: lse in units of log 2, +inf where the row sees nothing, with the bits of
// +inf turned so that the zeros that are read behind the last row stand for it, too;
// and -delta.
constexpr uint32_t kInfinity = 0x7f800000u;
struct Stats {
  float *turned_lse2, *minus_delta;
  __host__ __device__ Stats(float *at, int64_t tokens, int64_t heads)
      : turned_lse2(at), minus_delta(at + tokens * heads) {}
};
__device__ __forceinline__ float turned(float lse2) {
  return __uint_as_float(__float_as_uint(lse2) ^ kInfinity);
}

// Whether workgroups of 128 rows would leave CUs without one, or in float32, which
// the matrix cores bound, with one more than others: then two groups of waves share
// the keys of 64 rows.  (One sequence of 1466 keys, 8 heads of 96 in float32 93 us for
// 155, in bfloat16 25 for 29; of 2 x 2000 rows, 16 heads of 128, which 400 workgroups
// hold, 302 for 438 and 80 for 59.)
template <typename T>
inline bool few_tiles(int64_t tokens, int heads) {
  return tokens / 128 * heads < (sizeof(typename T::S) == 4 ? 512 : 256);
}

// Few rows that see many keys, in fewer heads than there are CUs for two of: no lone
// wave walks all the keys then.  (32 sequences of 20 rows after 1000 keys, 8 heads of
// 64: 51 us for 105 in float32, 19 for 39 in bfloat16; of 4 of 8 rows after 4000, 8
// heads of 128 the gradient 449 for 672 and 93 for 274.  256 sequences fill the card
// with waves: 302 for 692 the other way round.)  One workgroup walks all keys of its
// rows: one sequence of 16 after 100000, 8 heads of 128, which leaves most CUs without
// work, takes 7.6 ms in float32 and 1.6 in bfloat16.
inline bool few_of_long(int64_t batch, int heads, int64_t kv_tokens) {
  return kv_tokens / batch > 256 && batch * heads <= 512;
}

// Workgroups for that many items; each takes those a grid apart.
inline uint32_t grid_of(int64_t items) {
  return (uint32_t)(items < (1 << 22) ? items : 1 << 22);
}

}  // namespace dlrm
