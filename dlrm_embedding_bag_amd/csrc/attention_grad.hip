// attention_grad.hip -- the gradient of attention over packed sequences.
//
// With p[i, j] = exp(scale q[i] . k[j] - lse[i]), delta[i] = grad[i] . out[i] and
//   ds[i, j] = p[i, j] (grad[i] . v[j] - delta[i])
// over the keys that a row sees:
//   dq[i] = scale sum_j ds[i, j] k[j]
//   dk[j] = scale sum_i ds[i, j] q[i]     dv[j] = sum_i p[i, j] grad[i]
// where the sums of dk and dv run over the heads that share a key head too.
//
// Two kernels, so that every sum has one owner and one order (no atomics): a
// workgroup of the first owns rows and walks the keys, and leaves delta and lse
// side by side for the second, whose workgroups own keys and walk rows and heads.
// The scores are made twice for that: seven products of scores' size instead of
// five.  (Three sequences of up to 5000 rows, 32 heads of 128 in bfloat16: 570 us and
// 900 to 930, 680 TFLOP/s of the five products, 950 of the seven.)  Both keep scores
// transposed or not so that p and ds, made in registers, are operands of the next product
// where they stand, as in the forward pass; for bfloat16 rows both are rounded to bfloat16
// for it, which the matrix cores take at many times the rate of float32.
#include <math.h>

#include "attention_common.hpp"

namespace dlrm {
namespace {

template <typename T>
__device__ __forceinline__ float dot(const Operand<T> &a, const Operand<T> &b, float sum) {
  if constexpr (sizeof(typename T::S) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      sum = __builtin_fmaf(a.v[e >> 2][e & 3], b.v[e >> 2][e & 3], sum);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = __builtin_fmaf(bf16_lo(a.v[e]), bf16_lo(b.v[e]), sum);
      sum = __builtin_fmaf(bf16_hi(a.v[e]), bf16_hi(b.v[e]), sum);
    }
  }
  return sum;
}

// Rows: dq, and the rows' statistics.  GROUPS groups of WAVES waves hold the same rows
// and take every GROUPS-th tile of keys, as in the forward pass.
template <typename T, int DP, int WAVES, int BN, int GROUPS>
__global__ __launch_bounds__(WAVES *GROUPS *kWave, (waves_a_simd<T, DP>)) void grad_rows_kernel(AttentionGradParams p,
                                                                 float *ws, int64_t items) {
  using S = typename T::S;
  using L = LdsTile<T, BN, DP>;
  constexpr int BM = WAVES * 32, KT = BN / 32, STEPS = DP / 16, DT = DP / 32;
  constexpr int AHEAD = sizeof(S) == 2 ? 4 : 2;
  constexpr int SECOND = WAVES > 1 ? L::SIZE : 1;   // a lone wave has one buffer
  __shared__ u32x4_t k0s[GROUPS * L::SIZE], v0s[GROUPS * L::SIZE];
  __shared__ u32x4_t k1s[GROUPS * SECOND], v1s[GROUPS * SECOND];
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
    const int64_t row = (int64_t)t.row + mine;
    const bool there = mine < t.left;
    if (t.sequence < 0) {
      if (there && half == 0 && part == 0 && p.fill & 1) {
        S *dq = (S *)p.dq.data + row * p.dq.token + head * p.dq.head;
        for (int d = 0; d < dim; ++d) dq[d] = 0;
      }
      continue;
    }
    const Range keys = p.kv_offsets ? rows_of(p.kv_offsets, p.batch, p.kv_tokens, t.sequence)
                                    : Range{t.first, t.row - t.first + t.left};
    const SeenKeys seen(p.causal, keys.count, t.left, BM, wave, 32);
    const int seen_keys = seen.by(mine);
    const int count = seen.tile_any / BN + (seen.tile_any % BN != 0);
    const int kv_head = head / p.group;

    Operand<T> q[STEPS], g[STEPS];
    float delta = 0.0f;
    {
      const MemoryRow<T> qs((const S *)p.q.data + t.row * p.q.token + head * p.q.head, p.q.token,
                            t.left, dim, mine);
      const MemoryRow<T> gs((const S *)p.grad.data + t.row * p.grad.token + head * p.grad.head,
                            p.grad.token, t.left, dim, mine);
      const MemoryRow<T> os((const S *)p.out.data + t.row * p.out.token + head * p.out.head,
                            p.out.token, t.left, dim, mine);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int at = s * 16 + half * 8;
        q[s] = qs.load(at);
        g[s] = gs.load(at);
        delta = dot<T>(g[s], os.load(at), delta);
      }
    }
    delta += __uint_as_float(lane_xor<32>(__float_as_uint(delta)));
    float lse2 = there ? p.lse[row * p.heads + head] * kLog2e : INFINITY;
    if (lse2 == -INFINITY) lse2 = INFINITY;
    if (there && half == 0 && part == 0) {
      const Stats stats(ws, p.tokens, p.heads);
      stats.turned_lse2[head * p.tokens + row] = turned(lse2);
      stats.minus_delta[head * p.tokens + row] = -delta;
    }

    f32x16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16_t{};
    kload.start((const S *)p.k.data + keys.first * p.k.token + kv_head * p.k.head, keys.count);
    vload.start((const S *)p.v.data + keys.first * p.v.token + kv_head * p.v.head, keys.count);
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
      const int left = seen_keys - base - half * 4;
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        f32x16_t s = f32x16_t{}, dp = f32x16_t{};
        in_order<T, 2 * STEPS, AHEAD, true>(
            [&](int i) { return by_row.read(i % 2 ? v : k, j * 32, i / 2); },
            [&](int i, const Operand<T> &a) {
              if (i % 2)
                dp = multiply(a, g[i / 2], dp);
              else
                s = multiply(a, q[i / 2], s);
            });
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse2)) * (dp[i] - delta);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j * 32 + row_of(i, 0) >= left) s[i] = 0.0f;
        }
        const Operand<T> w[2] = {operand_of<T>(s, 0), operand_of<T>(s, 1)};
        in_order<T, 2 * DT, AHEAD, true>(
            [&](int i) { return by_column.read(k, j * 32 + i / DT * 16, i % DT); },
            [&](int i, const Operand<T> &a) { o[i % DT] = multiply(a, w[i / DT], o[i % DT]); });
      }
    };
    if constexpr (WAVES == 1) {
      for (int n = 0; n < rounds; ++n) {
        fill(k0, v0);
        landed();
        work(k0, v0, n);
        landed();
      }
    } else {
      if (rounds > 0) fill(k0, v0);
      for (int n = 0; n < rounds; n += 2) {
        landed();
        if (n + 1 < rounds) fill(k1, v1);
        work(k0, v0, n);
        if (n + 1 < rounds) {
          landed();
          if (n + 2 < rounds) fill(k0, v0);
          work(k1, v1, n + 1);
        }
      }
      landed();
    }
    if constexpr (GROUPS == 2) {
      const Meeting<WAVES, L::SIZE> meeting{
          {(LdsChunks)k0s, (LdsChunks)v0s, (LdsChunks)k1s, (LdsChunks)v1s}, wave * kWave + lane};
      if (part == 1) {
#pragma unroll
        for (int d = 0; d < DT; ++d) meeting.put(d, o[d]);
      }
      landed();
      if (part == 0) {
#pragma unroll
        for (int d = 0; d < DT; ++d) meeting.add(d, o[d]);
      }
      landed();
      if (part == 1) continue;
    }
    MemoryRow<T>((S *)p.dq.data + t.row * p.dq.token + head * p.dq.head, p.dq.token, t.left, dim,
                 mine)
        .store(o, p.scale, half);
  }
}

// The statistics of a tile's rows, 64 a load; zeros behind the last row.
template <int BN, int WAVES>
__device__ __forceinline__ void fill_stats(LdsFloats lds, const Stats &stats, int64_t at, int rows,
                                           int wave, int lane) {
  static_assert(BN <= kWave);
  const int n = rows < BN ? rows : BN;
  if (wave == 0) load_to_lds(buffer_of(stats.turned_lse2 + at, n * 4), lane * 4, lds);
  if (wave == WAVES - 1) load_to_lds(buffer_of(stats.minus_delta + at, n * 4), lane * 4, lds + kWave);
}

// Keys: dk and dv.  A lane holds one key of its wave's 32.  GROUPS groups of WAVES
// waves hold the same keys and take every GROUPS-th tile of rows, each from buffers
// of its own; their sums meet in LDS at the end.  A key that many rows see makes a
// long workgroup, and there are few of them (one for 128 keys of a key head): half
// as long, they spread evenly over the CUs.
template <typename T, int DP, int WAVES, int BN, int GROUPS>
__global__ __launch_bounds__(WAVES *GROUPS *kWave, (waves_a_simd<T, DP>)) void grad_keys_kernel(AttentionGradParams p,
                                                                 float *ws, int kv_heads,
                                                                 int64_t items) {
  using S = typename T::S;
  using L = LdsTile<T, BN, DP>;
  constexpr int BM = WAVES * 32, QT = BN / 32, STEPS = DP / 16, DT = DP / 32;
  constexpr int AHEAD = 1;
  constexpr int SECOND = WAVES > 1 ? L::SIZE : 1;   // a lone wave has one buffer
  __shared__ u32x4_t q0s[GROUPS * L::SIZE], g0s[GROUPS * L::SIZE];
  __shared__ u32x4_t q1s[GROUPS * SECOND], g1s[GROUPS * SECOND];
  __shared__ float s0s[GROUPS * 2 * kWave], s1s[GROUPS * 2 * kWave];
  const int lane = threadIdx.x % kWave, half = lane >> 5;
  const int wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int part = GROUPS > 1 ? wave_of_all / WAVES : 0, wave = wave_of_all - part * WAVES;
  const LdsChunks q0 = (LdsChunks)q0s, g0 = (LdsChunks)g0s, q1 = (LdsChunks)q1s,
                  g1 = (LdsChunks)g1s;
  const LdsFloats s0 = (LdsFloats)s0s, s1 = (LdsFloats)s1s;
  TileLoad<T, BN, DP, WAVES> qload(wave, lane, p.q.token, p.dim);
  TileLoad<T, BN, DP, WAVES> gload(wave, lane, p.grad.token, p.dim);
  ReadRows<T, BN, DP> by_row(lane);
  ReadColumns<T, BN, DP> by_column(lane);
  const float c = p.scale * kLog2e;
  const int32_t *key_offsets = p.kv_offsets ? p.kv_offsets : p.offsets;
  const Stats stats(ws, p.tokens, p.heads);
  // (the group's buffers: their size is a power of two beyond what keys reach)
  by_row.place += part * L::SIZE * 16;
  by_column.place += part * L::SIZE * 16;
  // of the lane's first four rows; the others are 8 apart
  const uint32_t by_stat = half * 16 + part * 2 * kWave * 4;

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int dim = in_loop(p.dim);
    // (the first keys, which most rows see, come first)
    const int64_t tiles = tile_count(p.kv_tokens, p.batch, BM);
    const Item at = item_of(item, tiles, kv_heads);
    const int kv_head = at.head;
    const Tile t = find_tile(key_offsets, p.batch, p.kv_tokens, tiles - 1 - at.tile, BM);
    if (t.left <= 0) continue;
    const int mine = wave * 32 + (lane & 31);   // key of the tile
    if (t.sequence < 0) {
      if (mine < t.left && half == 0 && part == 0) {
        const int64_t key = (int64_t)t.row + mine;
        S *dk = (S *)p.dk.data + key * p.dk.token + kv_head * p.dk.head;
        S *dv = (S *)p.dv.data + key * p.dv.token + kv_head * p.dv.head;
        for (int d = 0; d < dim; ++d) {
          if (p.fill & 2) dk[d] = 0;
          if (p.fill & 4) dv[d] = 0;
        }
      }
      continue;
    }
    const Range rows = p.kv_offsets ? rows_of(p.offsets, p.batch, p.tokens, t.sequence)
                                    : Range{t.first, t.row - t.first + t.left};
    // the first row that sees a key of the tile: as far from the last row as the
    // key from the last key
    auto first_row = [&](int key) {
      const int r = p.causal ? rows.count - (t.left - key) : 0;
      return r < 0 ? 0 : r;
    };
    const int wave_key = wave * 32;
    const int wave_end = wave_key + 31 < t.left ? wave_key + 31 : t.left - 1;
    // (a wave without keys has nothing to see)
    const int wave_from = wave_key < t.left ? first_row(wave_key) : rows.count;
    const int wave_full = wave_key < t.left ? first_row(wave_end) : rows.count;
    const int from_row = mine < t.left ? first_row(mine) : rows.count;
    const int n0 = first_row(0) / BN;
    const int per_head = rows.count / BN + (rows.count % BN != 0) - n0;

    Operand<T> k[STEPS], v[STEPS];
    {
      const MemoryRow<T> ks((const S *)p.k.data + t.row * p.k.token + kv_head * p.k.head, p.k.token,
                            t.left, dim, mine);
      const MemoryRow<T> vs((const S *)p.v.data + t.row * p.v.token + kv_head * p.v.head, p.v.token,
                            t.left, dim, mine);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        k[s] = ks.load(s * 16 + half * 8);
        v[s] = vs.load(s * 16 + half * 8);
      }
    }
    f32x16_t ok[DT], ov[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) ok[d] = ov[d] = f32x16_t{};

    // tiles of rows, head by head of the group: the next to be asked for
    const int total = per_head > 0 ? per_head * p.group : 0;
    const int rounds = total / GROUPS + (total % GROUPS != 0);
    struct Place {
      int head, tile;
    };
    auto move = [&](Place &at, int n) __attribute__((always_inline)) {
      at.tile += n;
      while (at.tile >= per_head) {
        at.tile -= per_head;
        ++at.head;
      }
    };
    Place asked{0, 0}, at_work{0, 0};
    if (total) {
      move(asked, part);
      at_work = asked;
    }
    auto fill = [&](LdsChunks q, LdsChunks g, LdsFloats st) __attribute__((always_inline)) {
      if (asked.head >= p.group) return;
      const int skip = (n0 + asked.tile) * BN, left = rows.count - skip;
      const int64_t head = (int64_t)kv_head * p.group + asked.head, row = (int64_t)rows.first + skip;
      qload.start((const S *)p.q.data + row * p.q.token + head * p.q.head, left);
      gload.start((const S *)p.grad.data + row * p.grad.token + head * p.grad.head, left);
      qload.fill(q + part * L::SIZE, dim, wave);
      gload.fill(g + part * L::SIZE, dim, wave);
      fill_stats<BN, WAVES>(st + part * 2 * kWave, stats, head * p.tokens + row, left, wave, lane);
      move(asked, GROUPS);
    };
    auto work = [&](LdsChunks q, LdsChunks g, LdsFloats st) __attribute__((always_inline)) {
      if (at_work.head >= p.group) return;
      const int base = (n0 + at_work.tile) * BN;
      move(at_work, GROUPS);
      if (wave_from - base >= BN) return;
      const bool masked = base < wave_full;
#pragma unroll
      for (int j = 0; j < QT; ++j) {
        by_row.here();
        by_column.here();
        f32x16_t s = f32x16_t{}, dp;
        in_order<T, STEPS, AHEAD, false>([&](int i) { return by_row.read(q, j * 32, i); },
                                        [&](int i, const Operand<T> &a) { s = multiply(a, k[i], s); });
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const f32x4_t lse2 = lds_at<f32x4_t>((LdsBytes)st, by_stat + (j * 32 + i * 2) * 4);
          const f32x4_t from = lds_at<f32x4_t>((LdsBytes)st, by_stat + (kWave + j * 32 + i * 2) * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i + e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + e], c, -turned(lse2[e])));
            dp[i + e] = from[e];
          }
        }
        in_order<T, STEPS, AHEAD, false>(
            [&](int i) { return by_row.read(g, j * 32, i); },
            [&](int i, const Operand<T> &a) { dp = multiply(a, v[i], dp); });
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[i] *= s[i];
        if (masked) {
          const int from = from_row - base - half * 4;   // rows of the tile before it do not see the key
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j * 32 + row_of(i, 0) < from) s[i] = dp[i] = 0.0f;
        }
        const Operand<T> wp[2] = {operand_of<T>(s, 0), operand_of<T>(s, 1)};
        const Operand<T> wd[2] = {operand_of<T>(dp, 0), operand_of<T>(dp, 1)};
        in_order<T, 4 * DT, AHEAD, false>(
            [&](int i) { return by_column.read(i % 2 ? q : g, j * 32 + i / 2 / DT * 16, i / 2 % DT); },
            [&](int i, const Operand<T> &a) {
              const int h = i / 2 / DT, d = i / 2 % DT;
              if (i % 2)
                ok[d] = multiply(a, wd[h], ok[d]);
              else
                ov[d] = multiply(a, wp[h], ov[d]);
            });
      }
    };
    if constexpr (WAVES == 1) {
      for (int n = 0; n < rounds; ++n) {
        fill(q0, g0, s0);
        landed();
        work(q0, g0, s0);
        landed();
      }
    } else {
      if (rounds > 0) fill(q0, g0, s0);
      for (int n = 0; n < rounds; n += 2) {
        landed();
        if (n + 1 < rounds) fill(q1, g1, s1);
        work(q0, g0, s0);
        if (n + 1 < rounds) {
          landed();
          if (n + 2 < rounds) fill(q0, g0, s0);
          work(q1, g1, s1);
        }
      }
      landed();
    }
    if constexpr (GROUPS == 2) {
      static_assert(Meeting<WAVES, L::SIZE>::EACH * 4 >= 2 * DT);
      const Meeting<WAVES, L::SIZE> meeting{
          {(LdsChunks)q0s, (LdsChunks)g0s, (LdsChunks)q1s, (LdsChunks)g1s}, wave * kWave + lane};
      if (part == 1) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          meeting.put(d, ok[d]);
          meeting.put(DT + d, ov[d]);
        }
      }
      landed();
      if (part == 0) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          meeting.add(d, ok[d]);
          meeting.add(DT + d, ov[d]);
        }
      }
      landed();   // the buffers are free for the next item
    }
    if (part == 0) {
      MemoryRow<T>((S *)p.dk.data + t.row * p.dk.token + kv_head * p.dk.head, p.dk.token, t.left,
                   dim, mine)
          .store(ok, p.scale, half);
      MemoryRow<T>((S *)p.dv.data + t.row * p.dv.token + kv_head * p.dv.head, p.dv.token, t.left,
                   dim, mine)
          .store(ov, 1.0f, half);
    }
  }
}

template <typename T, int DP, int WAVES, int BN, int GROUPS>
hipError_t run_rows(const AttentionGradParams &p, float *ws, hipStream_t stream) {
  const int64_t items = tile_count(p.tokens, p.batch, WAVES * 32) * p.heads;
  launch_kernel(grad_rows_kernel<T, DP, WAVES, BN, GROUPS>, dim3(grid_of(items)),
                dim3(WAVES * GROUPS * kWave), 0, stream, p, ws, items);
  return hipGetLastError();
}

template <typename T, int DP, int WAVES, int BN, int GROUPS>
hipError_t run_keys(const AttentionGradParams &p, float *ws, hipStream_t stream) {
  const int kv_heads = p.heads / p.group;
  const int64_t items = tile_count(p.kv_tokens, p.batch, WAVES * 32) * kv_heads;
  launch_kernel(grad_keys_kernel<T, DP, WAVES, BN, GROUPS>, dim3(grid_of(items)),
                dim3(WAVES * GROUPS * kWave), 0, stream, p, ws, kv_heads, items);
  return hipGetLastError();
}

// Sequences of few rows take a wave each, and none waits for another (64 of 100
// rows, 8 heads of 64: 35 us for 40).  Else a workgroup takes 128 rows or keys, but
// 64 keys where that would leave CUs without one (2 x 2000 rows, two key heads of
// 128: 210 us for 261).
template <typename T, int DP>
hipError_t run(const AttentionGradParams &p, float *ws, hipStream_t stream) {
  constexpr int BN = sizeof(typename T::S) == 4 ? 32 : 64;
  const bool few = (p.tokens > p.kv_tokens ? p.tokens : p.kv_tokens) / p.batch <= 128;
  if (p.tokens) {
    const hipError_t e = few ? run_rows<T, DP, 1, 32, 1>(p, ws, stream)
                         : few_tiles<T>(p.tokens, p.heads)
                             ? run_rows<T, DP, 2, BN, 2>(p, ws, stream)
                             : run_rows<T, DP, 4, BN, 1>(p, ws, stream);
    if (e != hipSuccess) return e;
  }
  if (!p.kv_tokens) return hipSuccess;
  if (few) return run_keys<T, DP, 1, 32, 1>(p, ws, stream);
  const int64_t wide = p.kv_tokens / 128 * (p.heads / p.group);
  if constexpr (DP == 32) {
    return run_keys<T, DP, 4, BN, 1>(p, ws, stream);
  } else {
    if constexpr (sizeof(typename T::S) == 2)
      if (wide >= 256) return run_keys<T, DP, 4, BN, 2>(p, ws, stream);
    return run_keys<T, DP, 2, BN, 2>(p, ws, stream);
  }
}

template <typename T>
hipError_t by_dim(const AttentionGradParams &p, float *ws, hipStream_t stream) {
  if (p.dim <= 32) return run<T, 32>(p, ws, stream);
  if (p.dim <= 64) return run<T, 64>(p, ws, stream);
  if (p.dim <= 96) return run<T, 96>(p, ws, stream);
  return run<T, 128>(p, ws, stream);
}

}  // namespace

size_t attention_grad_workspace(int64_t tokens, int heads) {
  return (size_t)tokens * heads * 2 * sizeof(float);
}

hipError_t launch_attention_grad(const AttentionGradParams &p, int dtype, void *workspace,
                                 hipStream_t stream) {
  // tiles of 16 rows for sequences of few (8 heads, the mean of their rows: in float32
  // of 64 elements 10 135 us for 214, 40 84 for 101; of 128 10 385 for 535, 40 203 for
  // 210; in bfloat16 of 128 10 169 for 244, 24 94 for 110, but 94 for 78 where all heads
  // share a key head's)
  if (p.tokens / p.batch <= (dtype == kF32 ? 40 : 16) &&
      !few_of_long(p.batch, p.heads, p.kv_tokens))
    return launch_attention_grad_short(p, dtype, workspace, stream);
  float *ws = (float *)workspace;
  return dtype == kF32 ? by_dim<F32>(p, ws, stream) : by_dim<BF16>(p, ws, stream);
}

}  // namespace dlrm
