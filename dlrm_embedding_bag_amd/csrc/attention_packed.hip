// attention_packed.hip -- attention over packed sequences.
//
//   s[i, j] = scale q[i] . k[j]   for the keys j that row i sees
//   out[i]  = sum_j exp(s[i, j] - lse[i]) v[j],   lse[i] = log sum_j exp(s[i, j])
//
// One pass over the keys with the running maximum m and sum l of each row's
// exponentials, in float32: a larger maximum scales what has been added.  A wave
// holds 32 rows, one for each lane of a half, and makes the transposed scores
// s^T = k q^T, so that a row's exponentials stay in its own two lanes and are
// the operand of out^T += v^T p^T without leaving the registers; keys and values
// pass through LDS, the next tile on its way while one is worked on.
//
// For bfloat16 rows the weights are rounded to bfloat16, which a library's product takes
// at nine times the rate of float32 (1400 for 154 TFLOP/s); their sum l takes them whole.
// (Against 64 bits the prompts' outputs are off by 0.0021 of their size, by 0.0016 where
// nothing but they themselves is rounded.)
//
// In bfloat16 of 128 elements the matrix cores are busy 48% of the time; between a wave's
// products stand its exponentials and its reads of LDS, and two waves a SIMD cover each
// other.  (Four prompts of up to 6500 rows, 32 heads: 800 to 850 us by card and run, 1000
// to 940 TFLOP/s; a single wave a SIMD with 64 rows, which halves the reads, 1207.  In
// float32 four of 1500 to 3000 rows 118 TFLOP/s.)
#include <math.h>

#include "attention_forward.hpp"

namespace dlrm {
namespace {

// GROUPS groups of WAVES waves hold the same rows and take every GROUPS-th tile of keys,
// each from buffers of its own; their sums meet in LDS at the end.
template <typename T, int DP, int WAVES, int BN, int GROUPS>
__global__ __launch_bounds__(WAVES *GROUPS *kWave, 2) void attention_kernel(AttentionParams p,
                                                                         int64_t items) {
  using S = typename T::S;
  using L = LdsTile<T, BN, DP>;
  constexpr int BM = WAVES * 32, KT = BN / 32, STEPS = DP / 16, DT = DP / 32;
  constexpr int AHEAD = sizeof(S) == 2 ? 4 : 2;
  constexpr int SECOND = WAVES > 1 ? L::SIZE : 1;   // a lone wave has one buffer
  __shared__ u32x4_t k0s[GROUPS * L::SIZE], v0s[GROUPS * L::SIZE];
  __shared__ u32x4_t k1s[GROUPS * SECOND], v1s[GROUPS * SECOND];
  __shared__ int found[WAVES * GROUPS];
  __shared__ float whole[GROUPS > 1 ? 2 * WAVES * kWave : 1];
  const int lane = threadIdx.x % kWave, half = lane >> 5;
  const int wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int part = GROUPS > 1 ? wave_of_all / WAVES : 0, wave = wave_of_all - part * WAVES;
  const LdsChunks k0 = (LdsChunks)k0s + part * L::SIZE, v0 = (LdsChunks)v0s + part * L::SIZE;
  const LdsChunks k1 = (LdsChunks)k1s + part * L::SIZE, v1 = (LdsChunks)v1s + part * L::SIZE;
  TileLoad<T, BN, DP, WAVES> kload(wave, lane, p.k.token, p.dim);
  TileLoad<T, BN, DP, WAVES> vload(wave, lane, p.v.token, p.dim);
  const ReadRows<T, BN, DP> by_row(lane);
  const ReadColumns<T, BN, DP> by_column(lane);
  const float c = p.scale * kLog2e;

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int dim = in_loop(p.dim);
    const int64_t tiles = tile_count(p.tokens, p.batch, BM);
    constexpr bool PAIRS = 4 * GROUPS * L::SIZE * 16 <= 80 << 10;   // as its LDS allows
    const bool by_work = WAVES > 1 && in_order_of_work(items, p.batch, p.kv_tokens);
    const Item at = item_of(by_work ? pair_up<PAIRS>(item, items) : item, tiles, p.heads);
    const int head = at.head;
    const Tile t = by_work ? tile_of_rank<BM>(p.offsets, p.kv_offsets, p.batch, p.tokens,
                                              p.kv_tokens, p.causal, (int)(tiles - 1 - at.tile))
                           : find_tile(p.offsets, p.batch, p.tokens, at.tile, BM);
    if (t.left <= 0) continue;
    const int mine = wave * 32 + (lane & 31);   // row of the tile
    if (t.sequence < 0) {
      if (mine < t.left && half == 0 && part == 0) put_nothing<T>(p, (int64_t)t.row + mine, head);
      continue;
    }
    const Range keys = p.kv_offsets ? rows_of(p.kv_offsets, p.batch, p.kv_tokens, t.sequence)
                                    : Range{t.first, t.row - t.first + t.left};
    const SeenKeys seen(p.causal, keys.count, t.left, BM, wave, 32);
    const int seen_keys = seen.by(mine);
    const int count = seen.tile_any / BN + (seen.tile_any % BN != 0);
    const int kv_head = head / p.group;
    const S *vbase = (const S *)p.v.data + keys.first * p.v.token + kv_head * p.v.head;
    Operand<T> q[STEPS];
    {
      const MemoryRow<T> from((const S *)p.q.data + t.row * p.q.token + head * p.q.head, p.q.token,
                              t.left, dim, mine);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) q[s] = from.load(s * 16 + half * 8);
    }
    f32x16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16_t{};
    float m = -INFINITY, l = 0.0f;
    int loose = -1;   // the first round of tiles whose values are not all added

    kload.start((const S *)p.k.data + keys.first * p.k.token + kv_head * p.k.head, keys.count);
    vload.start(vbase, keys.count);
    kload.skip(part * BN);
    vload.skip(part * BN);
    const int rounds = count / GROUPS + (count % GROUPS != 0);
    auto fill = [&](LdsChunks k, LdsChunks v) __attribute__((always_inline)) {
      if (GROUPS > 1 && kload.left <= 0) return;
      kload.fill(k, dim, wave);
      vload.fill(v, dim, wave);
      kload.skip((GROUPS - 1) * BN);
      vload.skip((GROUPS - 1) * BN);
    };
    auto work = [&](LdsChunks k, LdsChunks v, int n) __attribute__((always_inline)) {
      const int base = (n * GROUPS + part) * BN;
      if (base >= seen.wave_any) return;
      const bool masked = seen.wave_all - base < BN;
      f32x16_t s[KT];
#pragma unroll
      for (int j = 0; j < KT; ++j) s[j] = f32x16_t{};
      in_order<T, KT * STEPS, AHEAD, true>(
          [&](int i) { return by_row.read(k, i % KT * 32, i / KT); },
          [&](int i, const Operand<T> &a) { s[i % KT] = multiply(a, q[i / KT], s[i % KT]); });
      if (masked) {
        const int left = seen_keys - base - half * 4;
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j * 32 + row_of(i, 0) >= left) s[j][i] = -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[j][i]);
      top = fmaxf(top, __uint_as_float(lane_xor<32>(__float_as_uint(top))));
      const float next = fmaxf(m, top * c);
      if (__any(next > m + kSlack)) {
        // (a row that has seen nothing has m -inf and nothing to scale)
        const bool mine = next > m + kSlack;   // (a row does not follow another's)
        const float back = mine ? __builtin_amdgcn_exp2f(m - next) : 1.0f;
        l *= back;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= back;
        m = mine ? next : m;
      }
      const float from = m == -INFINITY ? 0.0f : m;
      // the weights of 16 keys at a time, those of the next 16 between the products
      auto weigh = [&](int i) __attribute__((always_inline)) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 16][i % 16], c, -from));
        s[i / 16][i % 16] = x;
        l += x;
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) weigh(i);
      Operand<T> w;
      in_order<T, BN / 16 * DT, AHEAD, false>(
          [&](int i) { return by_column.read(v, i / DT * 16, i % DT); },
          [&](int i, const Operand<T> &a) {
            const int j = i / DT, d = i % DT;
            if (d == 0) w = operand_of<T>(s[j / 2], j % 2);
            o[d] = multiply(a, w, o[d]);
            if (j + 1 < BN / 16) {
#pragma unroll
              for (int e = d * 8 / DT; e < (d + 1) * 8 / DT; ++e) weigh(8 * (j + 1) + e);
            }
          });
    };
    // A value that is not finite must not reach the rows that do not see it, and
    // zero times it is not zero: from the first tile on that some row does not see
    // whole, such values are left out, and added after the last tile.  (Rows of values
    // that repeat or overlap stand behind the last key too, where others are zeros.)
    auto round_of = [&](LdsChunks k, LdsChunks v, int n) __attribute__((always_inline)) {
      if ((p.causal || p.v.token < dim) && seen.tile_all - n * GROUPS * BN < GROUPS * BN &&
          clean<T, L::SIZE, WAVES, GROUPS>(v, (n * GROUPS + part) * BN < keys.count, found, wave,
                                           part, lane))
        loose = loose < 0 ? n : loose;
      work(k, v, n);
    };

    if constexpr (WAVES == 1) {
      for (int n = 0; n < rounds; ++n) {
        fill(k0, v0);
        landed();
        round_of(k0, v0, n);
        landed();
      }
    } else {
      if (rounds > 0) fill(k0, v0);
      for (int n = 0; n < rounds; n += 2) {
        landed();
        if (n + 1 < rounds) fill(k1, v1);
        round_of(k0, v0, n);
        if (n + 1 < rounds) {
          landed();
          if (n + 2 < rounds) fill(k0, v0);
          round_of(k1, v1, n + 1);
        }
      }
      landed();  // nobody reads the tiles any more
    }
    if constexpr (GROUPS == 2) {
      const Meeting<WAVES, L::SIZE> meeting{
          {(LdsChunks)k0s, (LdsChunks)v0s, (LdsChunks)k1s, (LdsChunks)v1s}, wave * kWave + lane};
      float *const with = whole + 2 * (wave * kWave + lane);
      if (part == 1) {
#pragma unroll
        for (int d = 0; d < DT; ++d) meeting.put(d, o[d]);
        with[0] = m;
        with[1] = l;
      }
      landed();
      if (part == 0) {
        const float other = with[0], next = fmaxf(m, other);
        const float from = next == -INFINITY ? 0.0f : next;
        const float mine_by = __builtin_amdgcn_exp2f(m - from);
        const float other_by = __builtin_amdgcn_exp2f(other - from);
        l = l * mine_by + with[1] * other_by;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[d] *= mine_by;
          meeting.add(d, o[d], other_by);
        }
        m = next;
      }
      landed();   // the buffers are free for the next item
      if (part == 1) continue;
    }

    if (loose >= 0)
      add_others<T, DT>(o, vbase, p.v.token, dim, loose * GROUPS * BN, seen.wave_any, seen_keys, half);
    l += __uint_as_float(lane_xor<32>(__float_as_uint(l)));
    put_row<T, DT>(p, o, m, l, t, dim, mine, head, half);
  }
}

template <typename T, int DP, int WAVES, int BN, int GROUPS>
hipError_t run(const AttentionParams &p, hipStream_t stream) {
  const int64_t items = tile_count(p.tokens, p.batch, WAVES * 32) * p.heads;
  launch_kernel(attention_kernel<T, DP, WAVES, BN, GROUPS>, dim3(grid_of(items)),
                dim3(WAVES * GROUPS * kWave), 0, stream, p, items);
  return hipGetLastError();
}

template <typename T, int WAVES, int BN, int GROUPS>
hipError_t by_dim(const AttentionParams &p, hipStream_t stream) {
  if (p.dim <= 32) return run<T, 32, WAVES, BN, GROUPS>(p, stream);
  if (p.dim <= 64) return run<T, 64, WAVES, BN, GROUPS>(p, stream);
  if (p.dim <= 96) return run<T, 96, WAVES, BN, GROUPS>(p, stream);
  return run<T, 128, WAVES, BN, GROUPS>(p, stream);
}

// Sequences of few rows take a wave each, and none waits for another (64 of 100 rows,
// 8 heads of 64: 12 us for 17 in bfloat16, 23 for 38 in float32); else four waves.
template <typename T, int BN>
hipError_t by_size(const AttentionParams &p, hipStream_t stream) {
  if (p.tokens / p.batch <= 128 && !few_of_long(p.batch, p.heads, p.kv_tokens))
    return by_dim<T, 1, 32, 1>(p, stream);
  if (few_tiles<T>(p.tokens, p.heads)) return by_dim<T, 2, BN, 2>(p, stream);
  return by_dim<T, 4, BN, 1>(p, stream);
}

}  // namespace

// Kernels go by the means of a call's sequences, since offsets are not read on the host:
// a long sequence among many short ones is walked by their kernel (32 heads of 128 in
// bfloat16: one of 2000 rows 53 us, beside 64 of one row 189; one of 4000 150 and 193).
hipError_t launch_attention(const AttentionParams &p, int dtype, hipStream_t stream) {
  // tiles of 16 rows for sequences of few (8 heads, the mean of their rows: in float32
  // of 64 elements 10 42 us for 83, 40 26 for 35; in bfloat16 of 128 10 54 for 80, 40 23
  // for 27, 64 44 for 36 with two waves a SIMD)
  if (p.tokens / p.batch <= 40 && !few_of_long(p.batch, p.heads, p.kv_tokens))
    return launch_attention_short(p, dtype, stream);
  return dtype == kF32 ? by_size<F32, 32>(p, stream) : by_size<BF16, 64>(p, stream);
}

}  // namespace dlrm
