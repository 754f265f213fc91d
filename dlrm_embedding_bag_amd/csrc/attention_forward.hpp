// attention_forward.hpp -- internal: what the kernels of attention over packed
// sequences share.
#pragma once

#include "attention_common.hpp"

namespace dlrm {

// The running maximum is a reference for the exponentials, which may exceed 1: it
// follows a larger score only where that lies 2^kSlack above it, so that sums and
// outputs are seldom scaled (at every tile of most rows otherwise).
constexpr float kSlack = 8.0f;

// Sign bits of a word's elements that are not finite.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return sizeof(typename T::S) == 4 ? ((w & 0x7fffffffu) + 0x00800000u) & 0x80000000u
                                    : ((w & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
}

template <typename T>
__device__ __forceinline__ uint32_t finite(uint32_t w) {   // zeros in their place
  const uint32_t n = not_finite<T>(w);
  // a sign bit to all bits of its element
  return w & ~(sizeof(typename T::S) == 4 ? (n ? 0xffffffffu : 0u) : (n >> 15) * 0xffffu);
}

// A tile of values in LDS for each group of WAVES waves: whether one holds a value
// that is not finite, for all waves; if so it is zero there when this returns.  A group
// whose tile is not `there` has nothing to say: what its part of LDS holds was left by
// whoever had it before.
template <typename T, int SIZE, int WAVES, int GROUPS>
__device__ __forceinline__ bool clean(LdsChunks v, bool there, int *found, int wave, int part,
                                      int lane) {
  constexpr int EACH = SIZE / (WAVES * kWave);
  uint32_t others = 0;
  if (GROUPS == 1 || there) {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const u32x4_t w = v[(i * WAVES + wave) * kWave + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) others |= not_finite<T>(w[e]);
    }
  }
  const bool mine = __any(others != 0);
  if (lane == 0) found[part * WAVES + wave] = mine;
  landed();
  bool any = false;
#pragma unroll
  for (int w = 0; w < WAVES * GROUPS; ++w) any |= found[w] != 0;
  if (!uniform((int)any)) return false;
  for (int i = 0; i < EACH; ++i) {
    LdsChunks at = v + (i * WAVES + wave) * kWave + lane;
    u32x4_t w = *at;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = finite<T>(w[e]);
    *at = w;
  }
  landed();
  return true;
}

// The values that `clean` left out, from key `first` on, for a row that sees them
// (weights are above zero, so they add as they are).
template <typename T, int DT>
__device__ __forceinline__ void add_others(f32x16_t (&o)[DT], const typename T::S *values,
                                           int64_t stride, int dim, int first, int last, int seen,
                                           int half) {
  for (int j = first; j < last; ++j) {
    if (j >= seen) continue;
    const typename T::S *at = values + (int64_t)j * stride;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = d * 32 + row_of(i, half);
        const float x = e < dim ? load1<T>(at + e) : 0.0f;
        if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) o[d][i] += x;
      }
  }
}

// The logarithm of a row's whole, l relative to m.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) * kLn2 + logf(l);
}

// A lane's half of a row: its sums relative to m, l the row's whole.
template <typename T, int DT>
__device__ __forceinline__ void put_row(const AttentionParams &p, const f32x16_t (&o)[DT], float m,
                                        float l, const Tile &t, int dim, int mine, int head,
                                        int half) {
  using S = typename T::S;
  const MemoryRow<T> out((S *)p.out.data + t.row * p.out.token + head * p.out.head, p.out.token,
                         t.left, dim, mine);
  out.store(o, l > 0.0f || l != l ? 1.0f / l : 0.0f, half);
  if (p.lse && half == 0 && mine < t.left)
    p.lse[((int64_t)t.row + mine) * p.heads + head] = lse_of(m, l);
}

// A row outside all sequences.
template <typename T>
__device__ __forceinline__ void put_nothing(const AttentionParams &p, int64_t row, int head) {
  using S = typename T::S;
  S *out = (S *)p.out.data + row * p.out.token + head * p.out.head;
  if (p.fill & 1)
    for (int d = 0; d < p.dim; ++d) out[d] = 0;
  if (p.fill & 2) p.lse[row * p.heads + head] = -INFINITY;
}

}  // namespace dlrm
