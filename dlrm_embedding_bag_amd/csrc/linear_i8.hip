// linear_i8.hip -- linear layer of int8 operands with a scale for each row of
// A (token) and of W (channel), bias and activation in the store path:
//
//   C[m, n] = act(bias[n] + a_scale[m] w_scale[n] sum_k A[m, k] W[n, k])
//
// The sum is exact: int8 products accumulated in int32 by the matrix cores
// (v_mfma_i32_16x16x64_i8); K is limited so that it cannot overflow.  The
// sum is then rounded to float32, scaled, and rounded once more to C's type.
//
// W is fed as the first operand, so a lane's 4 accumulators are 4 consecutive
// columns of one row of C.  Rows may start at any byte (a K of odd length):
// global memory takes 16-byte loads at any address.
//
// Three kernels, by the number of rows and the rows' alignment (launch_typed):
//   few_rows   up to 64 rows: bound by reading W.  1 x 8192 x 8192: 13 us,
//              5.2 TB/s; 32 x 8192 x 8192: 18 us, 64 rows 25, the rest A's
//              reads from L2 (every workgroup reads all of A)
//   staged     rows on 16 bytes.  8192^3: 453 us, 2.4 POP/s at 2.1 GHz, the
//              matrix cores busy 55% of the cycles.  Power has a part in that
//              (500 us of uniform codes under sustained load, 416 of codes within
//              +-3, 326 of zeros), waits the other; 128 x 8192 x 8192: 16 us, W's bytes
//   gemm       any rows, through registers.  2048 x 512 x 415: 7.2 us;
//              4001 x 4099 x 4093: 175 us (4096^3 from rows on 16 bytes: 61): loads
//              that cross 16 bytes, one slab of them in flight.  64 x 64 tiles
//              walk k alone, so few tiles leave CUs idle: 2000 x 100 x 5001, 64
//              workgroups, 21 us
#include <math.h>

#include <type_traits>

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

constexpr int kBK = 128;          // bytes of k per LDS slab
constexpr int kChunks = kBK / 16;
constexpr int kXcds = 8;

__device__ __forceinline__ i32x4_t load16(const int8_t *p) {
  return (i32x4_t) * reinterpret_cast<const u32x4_u *>(p);
}

// The 16 bytes of a row of K from which k's chunk [k, k + 16) is taken: the
// chunk itself, or, where it reaches past the row, the row's last 16 bytes.
// The same bytes are taken of both operands; those before k are products that
// an earlier chunk has, so one operand, A, has them zeroed (by first_from).
// Rows shorter than 16 are read byte by byte, zeros past their end.
__device__ __forceinline__ i32x4_t load16_tail(const int8_t *row, int k, int K) {
  if (K >= 16) return load16(row + (k + 16 <= K ? k : K - 16));
  unsigned __int128 v = 0;
  for (int e = K - 1; e >= k; --e) v = v << 8 | (uint8_t)row[e];
  return __builtin_bit_cast(i32x4_t, v);
}
__device__ __forceinline__ i32x4_t first_from(i32x4_t v, int k, int K) {
  const int gone = K >= 16 ? k + 16 - K : 0;  // leading bytes that are not of the chunk
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int g = gone - 4 * d;
    v[d] = g <= 0 ? v[d] : g >= 4 ? 0 : v[d] & (int)(0xffffffffu << (8 * g));
  }
  return v;
}

// What the store path needs of four consecutive columns, loaded before the
// first of them is stored (bias 0 where there is none).
struct Columns {
  f32x4_t scale, bias;
};
__device__ __forceinline__ float column_scale(const LinearI8Params &p, int n) {
  return p.w_scale[n < p.N ? n : p.N - 1];
}
__device__ __forceinline__ float column_bias(const LinearI8Params &p, int n) {
  return p.bias ? p.bias[n < p.N ? n : p.N - 1] : 0.0f;
}
__device__ __forceinline__ float row_scale(const LinearI8Params &p, int m) {
  return p.a_scale[m < p.M ? m : p.M - 1];
}
__device__ __forceinline__ Columns columns(const LinearI8Params &p, int n) {
  Columns c;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c.scale[e] = column_scale(p, n + e);
    c.bias[e] = column_bias(p, n + e);
  }
  return c;
}

// Whether the product of two such scales stays in float32's normal range.
__device__ __forceinline__ bool tame(float s) {
  return fabsf(s) >= 0x1p-63f && fabsf(s) <= 0x1p63f;
}
__device__ __forceinline__ bool tame(const Columns &c) {
  bool all = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) all &= tame(c.scale[e]);
  return all;
}

// Four sums scaled, with bias and activation.  TAME scales: the sum to float32,
// the scales' product, the sum times it plus the bias, a rounding each.  Of other
// scales that product may leave float32's range though a sum of 10^6 brings it
// back, or though the sum is zero: such quads (so that a row's bits depend on
// nothing but the row) go by float64, which holds the product of any two
// float32, and are rounded at the end.
template <bool TAME>
__device__ __forceinline__ void finish_quad(const LinearI8Params &p, i32x4_t acc, float as,
                                            const Columns &col, float (&v)[4]) {
  const float floor = p.act == 1 ? 0.0f : -INFINITY;  // of ReLU, or none
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = __builtin_fmaf((float)acc[e], as * col.scale[e], col.bias[e]);
  if (!TAME && !(tame(as) && tame(col))) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = (float)__builtin_fma((double)acc[e], (double)as * (double)col.scale[e],
                                  (double)col.bias[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = v[e] <= floor ? floor : v[e];  // NaN (a row without a scale) stays
  if (p.act == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = 1.0f / (1.0f + expf(-v[e]));
  }
}

__device__ __forceinline__ void put_quad(float *c, const float (&v)[4]) {
  *reinterpret_cast<f32x4_u *>(c) = f32x4_u{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void put_quad(uint16_t *c, const float (&v)[4]) {
  *reinterpret_cast<u32x2_u *>(c) = u32x2_u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// Columns n.. of row m.
template <typename TO, bool TAME>
__device__ __forceinline__ void store_quad(const LinearI8Params &p, int m, int n, i32x4_t acc,
                                           float as, const Columns &col) {
  using SO = typename TO::S;
  if (m >= p.M) return;
  SO *c = (SO *)p.C + (int64_t)m * p.ldc + n;
  float v[4];
  finish_quad<TAME>(p, acc, as, col, v);
  if (n + 4 <= p.N) {
    put_quad(c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) store1<TO>(c + e, v[e]);
  }
}

// Calls store(TAME) for a wave's tile: a wave whose scales are all tame, as
// nearly all are, takes a path without tests (which cost 8192 x 3000 x 201 2 of
// its 30 us).
template <int FM, int FN, typename Store>
__device__ __forceinline__ void by_scales(const float (&as)[FM], const Columns (&col)[FN],
                                          Store store) {
  bool all = true;
#pragma unroll
  for (int i = 0; i < FM; ++i) all &= tame(as[i]);
#pragma unroll
  for (int j = 0; j < FN; ++j) all &= tame(col[j]);
  if (__all(all))
    store(std::true_type());
  else
    store(std::false_type());
}

// The accumulators of a wave whose tile begins at row m0, column n0.
template <typename TO, int FM, int FN>
__device__ __forceinline__ void store_tile(const LinearI8Params &p, int m0, int n0,
                                           const i32x4_t (&acc)[FM][FN]) {
  const int fr = threadIdx.x % 16, fc = threadIdx.x % kWave / 16;
  float as[FM];
  Columns col[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i) as[i] = row_scale(p, m0 + i * 16 + fr);
#pragma unroll
  for (int j = 0; j < FN; ++j) col[j] = columns(p, n0 + j * 16 + fc * 4);
  by_scales(as, col, [&](auto tame) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        store_quad<TO, decltype(tame)::value>(p, m0 + i * 16 + fr, n0 + j * 16 + fc * 4,
                                              acc[i][j], as[i], col[j]);
  });
}

// Tile of workgroup b: each XCD (workgroups are dealt to them in turn) takes
// a contiguous run of tiles, and a run goes down columns of kGroup row tiles,
// so that the tiles in flight on an XCD share rows of A and of W in its L2.
__device__ __forceinline__ void tile_of(int b, int tm, int tn, int &im, int &in) {
  constexpr int kGroup = 8;
  const int all = tm * tn, q = all / kXcds, r = all % kXcds;
  const int x = b % kXcds;
  const int t = x * q + (x < r ? x : r) + b / kXcds;
  const int span = kGroup * tn;
  const int g = t / span, rest = t - g * span;
  const int rows = tm - g * kGroup < kGroup ? tm - g * kGroup : kGroup;
  im = g * kGroup + rest % rows;
  in = rest / rows;
}

// BM x BN tile on GM x GN waves; slabs of 128 bytes of k go through registers
// to two LDS buffers (any alignment), D slabs ahead: few workgroups wait for
// memory at every slab (2000 x 100 x 5001: 32 us with one ahead, 24 with two, 21
// with three; 1000 x 1000 x 1001: 9.1, 8.7, 9.0), larger tiles want the
// registers (4000 x 2000 x 999: 24, 26, 36).  A row's 16-byte chunk c
// lies at place c ^ (row % 8) of its 128-byte row: the rows that a ds_read_b128
// touches start on different banks.
template <int BM, int BN, int GM, int GN, int D, typename TO>
__global__ __launch_bounds__(GM *GN *kWave) void gemm_kernel(LinearI8Params p, int tm, int tn) {
  constexpr int T = GM * GN * kWave;
  constexpr int FM = BM / GM / 16, FN = BN / GN / 16;
  constexpr int CA = BM * kChunks / T, CB = BN * kChunks / T;
  __shared__ i32x4_t lds[2][(BM + BN) * kChunks];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int wm = wave / GN, wn = wave % GN;
  int im, in;
  tile_of(blockIdx.x, tm, tn, im, in);
  const int m0 = im * BM, n0 = in * BN;
  const int crow = tid / kChunks, cch = tid % kChunks;

  i32x4_t ra[D][CA], rb[D][CB];
  const int whole = p.K / kBK, slabs = (p.K + kBK - 1) / kBK;
  auto load = [&](int slab, i32x4_t (&ra)[CA], i32x4_t (&rb)[CB], auto inner) {
    const int k = slab * kBK + cch * 16;
    const bool full = inner || slab < whole;
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int m = m0 + crow + i * (T / kChunks);
      const int8_t *row = p.A + (int64_t)(m < p.M ? m : p.M - 1) * p.lda;
      ra[i] = full ? load16(row + k) : first_from(load16_tail(row, k, p.K), k, p.K);
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int n = n0 + crow + i * (T / kChunks);
      const int8_t *row = p.W + (int64_t)(n < p.N ? n : p.N - 1) * p.ldw;
      rb[i] = full ? load16(row + k) : load16_tail(row, k, p.K);
    }
  };
  auto stage = [&](int buf, const i32x4_t (&ra)[CA], const i32x4_t (&rb)[CB]) {
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int r = crow + i * (T / kChunks);
      lds[buf][r * kChunks + (cch ^ (r & 7))] = ra[i];
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int r = crow + i * (T / kChunks);
      lds[buf][(BM + r) * kChunks + (cch ^ (r & 7))] = rb[i];
    }
  };

  i32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

  const int fr = lane % 16, fc = lane / 16;
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < slabs) load(d, ra[d], rb[d], std::false_type());
  stage(0, ra[0], rb[0]);
  // Slab s, in LDS; register slot u held it and takes slab s + D.  `inner`: that
  // one is whole.
  auto step = [&](int s, auto slot, auto inner) {
    constexpr int U = decltype(slot)::value, NEXT = (U + 1) % D;
    __syncthreads();
    if (inner || s + D < slabs) load(s + D, ra[U], rb[U], inner);
    const i32x4_t *a = lds[s & 1] + (wm * (BM / GM)) * kChunks;
    const i32x4_t *b = lds[s & 1] + (BM + wn * (BN / GN)) * kChunks;
#pragma unroll
    for (int h = 0; h < kBK / 64; ++h) {
      i32x4_t fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = a[(i * 16 + fr) * kChunks + ((h * 4 + fc) ^ (fr & 7))];
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = b[(j * 16 + fr) * kChunks + ((h * 4 + fc) ^ (fr & 7))];
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    if (inner || s + 1 < slabs) stage((s + 1) & 1, ra[NEXT], rb[NEXT]);
  };
  auto steps = [&](int s, auto inner) {
    step(s, std::integral_constant<int, 0>(), inner);
    if constexpr (D > 1)
      if (inner || s + 1 < slabs) step(s + 1, std::integral_constant<int, 1>(), inner);
    if constexpr (D > 2)
      if (inner || s + 2 < slabs) step(s + 2, std::integral_constant<int, 2>(), inner);
  };
  static_assert(D >= 1 && D <= 3);
  int s = 0;
  for (; s + 2 * D <= whole; s += D) steps(s, std::true_type());
  for (; s < slabs; s += D) steps(s, std::false_type());
  store_tile<TO>(p, m0 + wm * (BM / GM), n0 + wn * (BN / GN), acc);
}

// Tiles of BM x BN on GM x GN waves for rows that start on 16 bytes: k in
// stages of ST bytes through four LDS buffers that the loads fill without
// registers.  While the matrix cores work on stage s from registers, its
// successor's operands are read from LDS into others, and stages s + 2 and
// s + 3 are on their way from memory into two more buffers; the fourth, that of
// stage s, takes stage s + 4.
// A tile's rows as a buffer, so that a load's address is a lane's own offset, kept
// for the whole loop, and one scalar that says how far k has come.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const int8_t *p) {
  // raw bytes, no stride; the last word is the format of 32-bit elements
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(p), 0, 0xffffffffu, 4 << 15);
}
// 16 bytes a lane, from memory to LDS: lane l's to lds[l].
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t lane_offset,
                                            int offset, i32x4_t *lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, lds, 16, lane_offset, offset, 0, 0);
}

// s_waitcnt's operand: no LDS access left, and at most `loads` loads.
constexpr int wait_for(int loads) { return 0x070 | (loads & 15) | (loads >> 4) << 14; }

template <int BM, int BN, int GM, int GN, int ST, typename TO>
__global__ __launch_bounds__(GM *GN *kWave) void staged_kernel(LinearI8Params p, int tm,
                                                                        int tn) {
  constexpr int WAVES = GM * GN, FM = BM / GM / 16, FN = BN / GN / 16, H = ST / 64;
  constexpr int C = ST / 16, R = kWave / C;            // chunks of a row, rows of a load
  constexpr int LOADS = (BM + BN) / (WAVES * R);       // of a wave, first those of A
  static_assert(BM % (WAVES * R) == 0 && BN % (WAVES * R) == 0 && LOADS * 2 < 64);
  __shared__ i32x4_t buf0[(BM + BN) * C], buf1[(BM + BN) * C], buf2[(BM + BN) * C],
      buf3[(BM + BN) * C];
  __shared__ float scales[BM + 2 * BN];  // of the rows, of the columns, and their bias
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / GN, wn = wave % GN;
  int im, in;
  tile_of(blockIdx.x, tm, tn, im, in);
  const int m0 = im * BM, n0 = in * BN;
  const int fr = lane % 16, fc = lane / 16;

  // Chunk c of row r lies at another place of the row, so that the 8 lanes that
  // read LDS together (8 rows, one chunk) start on different banks.
  auto place = [](int r, int c) { return c ^ (C == 8 ? r & 7 : r >> 1 & 3); };
  const auto abuf = buffer_of(p.A + (int64_t)m0 * p.lda);
  const auto wbuf = buffer_of(p.W + (int64_t)n0 * p.ldw);
  uint32_t from[LOADS];  // within the tile's rows
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = (i * WAVES + wave) * R + lane / C;  // of A, then of W
    const int c = place(r, lane % C);
    if (i < BM / (WAVES * R))
      from[i] = (uint32_t)(m0 + r < p.M ? r : p.M - 1 - m0) * (uint32_t)p.lda + c * 16;
    else
      from[i] =
          (uint32_t)(n0 + r - BM < p.N ? r - BM : p.N - 1 - n0) * (uint32_t)p.ldw + c * 16;
  }
  const int stages = p.K / ST;
  auto load = [&](i32x4_t *buf, int s) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      load_to_lds(i < BM / (WAVES * R) ? abuf : wbuf, from[i], s * ST,
                  buf + (i * WAVES + wave) * kWave);
  };
  auto read = [&](const i32x4_t *buf, i32x4_t (&fa)[H][FM], i32x4_t (&fb)[H][FN]) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int at = fr * C + place(fr, h * 4 + fc);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[h][j] = buf[(BM + (wn * FN + j) * 16) * C + at];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[h][i] = buf[(wm * FM + i) * 16 * C + at];
    }
  };

  i32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  auto multiply = [&](const i32x4_t (&fa)[FM], const i32x4_t (&fb)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
  };
  i32x4_t fa[2][H][FM], fb[2][H][FN];

  for (int i = threadIdx.x; i < BM + 2 * BN; i += WAVES * kWave)
    scales[i] = i < BM        ? row_scale(p, m0 + i)
                : i < BM + BN ? column_scale(p, n0 + i - BM)
                              : column_bias(p, n0 + i - BM - BN);
  if (stages > 0) load(buf0, 0);
  if (stages > 1) load(buf1, 1);
  if (stages > 2) load(buf2, 2);
  if (stages > 3) load(buf3, 3);
  __builtin_amdgcn_s_waitcnt(wait_for(0));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  if (stages > 0) read(buf0, fa[0], fb[0]);
  // Stage s, whose operands are in registers `now`; own is its buffer, next
  // that of stage s + 1.  `inner`: stages up to s + 4 follow.
  auto step = [&](int s, i32x4_t *own, const i32x4_t *next, int now, auto inner) {
    // own loads of stage s + 1 have landed (those of s + 2, s + 3 are younger),
    // and after the barrier everyone's have, and everyone holds stage s
    if (inner || s + 3 < stages)
      __builtin_amdgcn_s_waitcnt(wait_for(2 * LOADS));
    else
      __builtin_amdgcn_s_waitcnt(wait_for(0));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (inner || s + 4 < stages) load(own, s + 4);
    __builtin_amdgcn_sched_barrier(0);
    if (inner || s + 1 < stages) read(next, fa[now ^ 1], fb[now ^ 1]);
#pragma unroll
    for (int h = 0; h < H; ++h) multiply(fa[now][h], fb[now][h]);
    // reads from LDS between the products, the products' last third without
    constexpr int EACH = FM * FN / (FM + FN) > 2 ? 2 : 1;
#pragma unroll
    for (int q = 0; q < H * (FM + FN); ++q) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, EACH, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int s = 0;
  for (; s + 8 <= stages; s += 4) {
    step(s, buf0, buf1, 0, std::true_type());
    step(s + 1, buf1, buf2, 1, std::true_type());
    step(s + 2, buf2, buf3, 0, std::true_type());
    step(s + 3, buf3, buf0, 1, std::true_type());
  }
  for (; s < stages; s += 4) {
    step(s, buf0, buf1, 0, std::false_type());
    if (s + 1 < stages) step(s + 1, buf1, buf2, 1, std::false_type());
    if (s + 2 < stages) step(s + 2, buf2, buf3, 0, std::false_type());
    if (s + 3 < stages) step(s + 3, buf3, buf0, 1, std::false_type());
  }
  // what the stages leave of k, straight from memory
  for (int k = stages * ST + fc * 16; k - fc * 16 < p.K; k += 64) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = n0 + (wn * FN + j) * 16 + fr;
      fb[0][0][j] = load16_tail(p.W + (int64_t)(n < p.N ? n : p.N - 1) * p.ldw, k, p.K);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m0 + (wm * FM + i) * 16 + fr;
      fa[0][0][i] =
          first_from(load16_tail(p.A + (int64_t)(m < p.M ? m : p.M - 1) * p.lda, k, p.K), k, p.K);
    }
    multiply(fa[0][0], fb[0][0]);
  }
  Columns col[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = (wn * FN + j) * 16 + fc * 4 + e;
      col[j].scale[e] = scales[BM + n];
      col[j].bias[e] = scales[BM + BN + n];
    }
  }
  // 16 rows at a time go through LDS (the buffers are free: all waves hold the
  // last stage), so that a store takes whole pieces of a row, as long as the
  // wave's columns are; the products' own layout has 4 columns of 16 rows
  using SO = typename TO::S;
  constexpr int COLS = FN * 16, PITCH = COLS + 16 / (int)sizeof(SO);   // elements
  constexpr int UNIT = 16 / (int)sizeof(SO), UNITS = COLS / UNIT, ROWS = kWave / UNITS;
  SO *const slice = (SO *)(wave < WAVES / 2 ? buf0 : buf1) + wave % (WAVES / 2) * (16 * PITCH);
  static_assert(WAVES / 2 * 16 * PITCH * sizeof(SO) <= sizeof(buf0));
  const int nw = n0 + wn * COLS;
  float as[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) as[i] = scales[(wm * FM + i) * 16 + fr];
  by_scales(as, col, [&](auto tame) {
    constexpr bool TAME = decltype(tame)::value;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int mw = m0 + (wm * FM + i) * 16;
      if (nw + COLS <= p.N) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          float v[4];
          finish_quad<TAME>(p, acc[i][j], as[i], col[j], v);
          put_quad(slice + fr * PITCH + j * 16 + fc * 4, v);
        }
#pragma unroll
        for (int r = lane / UNITS; r < 16; r += ROWS) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t *>(slice + r * PITCH +
                                                               lane % UNITS * UNIT);
          if (mw + r < p.M)
            put16<false>((SO *)p.C + (int64_t)(mw + r) * p.ldc + nw + lane % UNITS * UNIT, v);
        }
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j)
          store_quad<TO, TAME>(p, mw + fr, nw + j * 16 + fc * 4, acc[i][j], as[i], col[j]);
      }
    }
  });
}

// Few rows, bound by reading W once: a workgroup takes 16 NF columns and all
// (up to 16 MF) rows; its 8 waves share k, 128 bytes at a time, with operands
// loaded straight into the matrix cores' layout, and add their partial tiles
// through LDS.  A wave keeps U steps' loads in flight all along: a step's
// registers are loaded again as soon as its products are issued.
constexpr int kFewWaves = 8;
template <int MF, int NF, int U, typename TO>
__global__ __launch_bounds__(kFewWaves *kWave) void few_rows_kernel(LinearI8Params p) {
  __shared__ i32x4_t part[kFewWaves][MF * NF][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int fr = lane % 16, fc = lane / 16;
  const int n0 = blockIdx.x * (16 * NF);
  const int8_t *wrow[NF], *arow[MF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const int n = n0 + j * 16 + fr;
    wrow[j] = p.W + (int64_t)(n < p.N ? n : p.N - 1) * p.ldw;
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = i * 16 + fr;
    arow[i] = p.A + (int64_t)(m < p.M ? m : p.M - 1) * p.lda;
  }
  // the four columns that this thread stores in the end, and their scales
  static_assert(MF * NF <= kFewWaves);
  const int sf = wave < MF * NF ? wave : 0;
  const int sm = sf / NF * 16 + fr, sn = n0 + sf % NF * 16 + fc * 4;
  const float as = row_scale(p, sm);
  const Columns col = columns(p, sn);
  i32x4_t acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

  // k goes in pairs of steps of 64 bytes, dealt to the waves in turn.  Rows
  // often lie a multiple of 4 KB apart, so that the 16 of a load share one L2
  // channel, and workgroups in step would all ask the same few: each begins at
  // another pair.
  const int pairs = p.K / 128;
  const int turn = pairs > 0 ? (int)(blockIdx.x / kXcds * 2 % pairs) : 0;
  const int mine = pairs > wave ? (pairs - wave + kFewWaves - 1) / kFewWaves * 2 : 0;  // steps
  i32x4_t w[U][NF], a[U][MF];
  auto load = [&](int i, i32x4_t (&w)[NF], i32x4_t (&a)[MF]) {
    int pair = i / 2 * kFewWaves + wave + turn;
    pair -= pair >= pairs ? pairs : 0;
    const int k = pair * 128 + i % 2 * 64 + fc * 16;
#pragma unroll
    for (int j = 0; j < NF; ++j) w[j] = load16(wrow[j] + k);
#pragma unroll
    for (int i = 0; i < MF; ++i) a[i] = load16(arow[i] + k);
  };
  auto multiply = [&](const i32x4_t (&w)[NF], const i32x4_t (&a)[MF]) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], a[i], acc[i][j], 0, 0, 0);
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < mine) load(u, w[u], a[u]);
  int i0 = 0;
  // (without a branch between loads, so that each wait is for the oldest alone)
  for (; i0 + 2 * U <= mine; i0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      multiply(w[u], a[u]);
      load(i0 + u + U, w[u], a[u]);
    }
  }
  for (; i0 < mine; i0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u < mine) multiply(w[u], a[u]);
      if (i0 + u + U < mine) load(i0 + u + U, w[u], a[u]);
    }
  }
  // what the pairs leave of k
  if (pairs * 128 < p.K && pairs % kFewWaves == wave) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = pairs * 128 + h * 64 + fc * 16;
#pragma unroll
      for (int j = 0; j < NF; ++j) w[h][j] = load16_tail(wrow[j], k, p.K);
#pragma unroll
      for (int i = 0; i < MF; ++i) a[h][i] = load16_tail(arow[i], k, p.K);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < MF; ++i)
        a[h][i] = first_from(a[h][i], pairs * 128 + h * 64 + fc * 16, p.K);
      multiply(w[h], a[h]);
    }
  }
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) part[wave][i * NF + j][lane] = acc[i][j];
  __syncthreads();
  if (threadIdx.x < MF * NF * kWave) {
    i32x4_t s = part[0][sf][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += part[w][sf][lane];
    store_quad<TO, false>(p, sm, sn, s, as, col);
  }
}

template <int BM, int BN, int GM, int GN, int D, typename TO>
void launch_tiles(const LinearI8Params &p, hipStream_t stream) {
  const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  launch_kernel(gemm_kernel<BM, BN, GM, GN, D, TO>, dim3((unsigned)(tm * tn)),
                dim3(GM * GN * kWave), 0, stream, p, tm, tn);
}

template <int BM, int BN, int GM, int GN, int ST, typename TO>
void launch_staged(const LinearI8Params &p, hipStream_t stream) {
  const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  launch_kernel(staged_kernel<BM, BN, GM, GN, ST, TO>, dim3((unsigned)(tm * tn)),
                dim3(GM * GN * kWave), 0, stream, p, tm, tn);
}

// Rows that the staged kernel takes: whole chunks, 256 of them within 32 bits.
bool staged_rows(const int8_t *p, int64_t ld) {
  return aligned16(p) && ld % 16 == 0 && ld < (int64_t)1 << 24;
}

template <int MF, int NF, int U, typename TO>
void launch_few(const LinearI8Params &p, hipStream_t stream) {
  launch_kernel(few_rows_kernel<MF, NF, U, TO>, dim3((p.N + 16 * NF - 1) / (16 * NF)),
                dim3(kFewWaves * kWave), 0, stream, p);
}

// Up to 64 rows few_rows, which is right for a few.  The tiles overtake it before
// that: N = K = 8192 takes it 18.4 us for 32 rows and 25.9 for 64, the staged
// kernel 15.9 for 65; of rows at any byte, N = 8192, K = 8191, it takes 40 us for 8,
// 60 for 32 and 88 for 64, the gemm 31 for 65.
// Tiles of 256 where they make more than half as many workgroups as CUs
// (3000 x 3000 x 3008: 44 us, 52 with 128, 55 with 64; 1024 x 8192 x 8192, 128
// of them: 93, 87, 96); of 128 where they make 256 (1000 x 4096 x 4096: 27 us,
// 30 with 64; 256 x 4096 x 4096, 64 of them: 21 and 10); else of 64.
template <typename TO>
hipError_t launch_typed(const LinearI8Params &p, hipStream_t stream) {
  const bool many = p.N >= 8192;  // columns: two 16-column fragments still make 256 workgroups
  if (p.M <= 64) {
    if (p.M <= 16)
      many ? launch_few<1, 2, 8, TO>(p, stream) : launch_few<1, 1, 8, TO>(p, stream);
    else if (p.M <= 32)
      many ? launch_few<2, 2, 8, TO>(p, stream) : launch_few<2, 1, 8, TO>(p, stream);
    else
      many ? launch_few<4, 2, 4, TO>(p, stream) : launch_few<4, 1, 4, TO>(p, stream);
    return hipGetLastError();
  }
  auto tiles = [&](int64_t b) { return (p.M + b - 1) / b * ((p.N + b - 1) / b); };
  const bool staged = staged_rows(p.A, p.lda) && staged_rows(p.W, p.ldw);
  if (tiles(256) > 128)
    staged ? launch_staged<256, 256, 2, 4, 64, TO>(p, stream)
           : launch_tiles<256, 256, 2, 4, 1, TO>(p, stream);
  else if (tiles(128) >= 256)
    staged ? launch_staged<128, 128, 2, 2, 64, TO>(p, stream)
           : launch_tiles<128, 128, 2, 2, 1, TO>(p, stream);
  else if (staged)
    launch_staged<64, 64, 2, 2, 128, TO>(p, stream);
  else if (p.K > 2048)
    launch_tiles<64, 64, 2, 2, 3, TO>(p, stream);
  else
    launch_tiles<64, 64, 2, 2, 2, TO>(p, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_i8(const LinearI8Params &p, int out_dtype, hipStream_t stream) {
  return out_dtype == kBF16 ? launch_typed<BF16>(p, stream) : launch_typed<F32>(p, stream);
}

}  // namespace dlrm
