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
// The scores' tile of 32 x 32 takes as long on the matrix cores (2 dim products
// of 32 x 32) as its exponentials on the vector units at dim 128, so two waves a
// SIMD cover each other.
#include <math.h>

#include "attention_common.hpp"

namespace dlrm {
namespace {

// Masks of the elements of a word that are not finite.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if constexpr (sizeof(typename T::S) == 4)
    return (w & 0x7f800000u) == 0x7f800000u ? 0xffffffffu : 0u;
  else
    return ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u) |
           ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u);
}
template <typename T>
constexpr int kWords = 8 * (int)sizeof(typename T::S) / 4;  // of an operand

template <typename T>
__device__ __forceinline__ uint32_t word_of(const Operand<T> &o, int i) {
  if constexpr (sizeof(typename T::S) == 4)
    return __float_as_uint(o.v[i >> 2][i & 3]);
  else
    return o.v[i];
}
template <typename T>
__device__ __forceinline__ void set_word(Operand<T> &o, int i, uint32_t w) {
  if constexpr (sizeof(typename T::S) == 4)
    o.v[i >> 2][i & 3] = __uint_as_float(w);
  else
    o.v[i] = w;
}
template <typename T>
__device__ __forceinline__ bool any_not_finite(const Operand<T> &o) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < kWords<T>; ++i) bad |= not_finite<T>(word_of<T>(o, i));
  return bad != 0;
}
// Its finite elements, zeros for the others.
template <typename T>
__device__ __forceinline__ Operand<T> finite_part(const Operand<T> &o) {
  Operand<T> r;
#pragma unroll
  for (int i = 0; i < kWords<T>; ++i)
    set_word<T>(r, i, word_of<T>(o, i) & ~not_finite<T>(word_of<T>(o, i)));
  return r;
}
// The element of slot `slot` if it is not finite (and `mine`), zeros elsewhere.
template <typename T>
__device__ __forceinline__ Operand<T> other_part(const Operand<T> &o, int slot, bool mine) {
  Operand<T> r;
  constexpr int E = 4 / (int)sizeof(typename T::S);
#pragma unroll
  for (int i = 0; i < kWords<T>; ++i) {
    const uint32_t w = word_of<T>(o, i);
    const uint32_t keep = E == 1 ? 0xffffffffu : slot & 1 ? 0xffff0000u : 0xffffu;
    set_word<T>(r, i, mine && slot / E == i ? w & not_finite<T>(w) & keep : 0u);
  }
  return r;
}

template <typename T, int DP, int WAVES, int BN>
__global__ __launch_bounds__(WAVES *kWave) void attention_kernel(AttentionParams p,
                                                                 int64_t items) {
  using S = typename T::S;
  using L = LdsTile<T, BN, DP>;
  constexpr int BM = WAVES * 32, KT = BN / 32, STEPS = DP / 16, DT = DP / 32;
  __shared__ u32x4_t k0[L::SIZE], v0[L::SIZE], k1[L::SIZE], v1[L::SIZE];
  const int lane = threadIdx.x % kWave, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const TileLoad<T, BN, DP, WAVES> kload(wave, lane, p.k.token, p.dim);
  const TileLoad<T, BN, DP, WAVES> vload(wave, lane, p.v.token, p.dim);
  const float c = p.scale * kLog2e;

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t tile = item / p.heads;
    const int head = (int)(item - tile * p.heads);
    const Tile t = find_tile(p.offsets, p.batch, p.tokens, tile, BM);
    if (t.row >= t.last) continue;
    const int64_t row = t.row + wave * 32 + (lane & 31);
    const bool there = row < t.last;
    S *out = (S *)p.out.data + row * p.out.token + head * p.out.head;
    if (t.sequence < 0) {
      if (there && half == 0 && p.fill & 1)
        for (int d = 0; d < p.dim; ++d) out[d] = 0;
      if (there && half == 0 && p.fill & 2) p.lse[row * p.heads + head] = -INFINITY;
      continue;
    }
    const KeyRange range = keys_of(p.offsets, p.kv_offsets, p.batch, p.kv_tokens, t);
    const SeenKeys seen(p.causal, range.count, t.last, t.row, BM, wave, row, there);
    const int64_t count = (seen.tile_any + BN - 1) / BN;
    const int kv_head = head / p.group;
    const S *kbase = (const S *)p.k.data + range.first * p.k.token + kv_head * p.k.head;
    const S *vbase = (const S *)p.v.data + range.first * p.v.token + kv_head * p.v.head;
    Operand<T> q[STEPS];
    {
      const S *at = (const S *)p.q.data + row * p.q.token + head * p.q.head;
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        q[s] = load_operand<T>(at, s * 16 + half * 8, p.dim, there);
    }
    f32x16_t o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16_t{};
    float m = -INFINITY, l = 0.0f;

    auto fill = [&](u32x4_t *k, u32x4_t *v, int64_t n) {
      kload.fill(k, kbase + n * BN * p.k.token, range.count - n * BN, p.k.token, p.dim, wave);
      vload.fill(v, vbase + n * BN * p.v.token, range.count - n * BN, p.v.token, p.dim, wave);
    };
    auto work = [&](const u32x4_t *k, const u32x4_t *v, int64_t n) {
      const int64_t base = n * BN;
      if (base >= seen.wave_any) return;
      const bool masked = base + BN > seen.wave_all;
      f32x16_t s[KT];
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        s[j] = f32x16_t{};
#pragma unroll
        for (int e = 0; e < STEPS; ++e)
          s[j] = multiply(read_rows<T, BN, DP>(k, j * 32, e, lane), q[e], s[j]);
      }
      if (masked) {
        const int left = (int)(seen.mine - base < BN ? seen.mine - base : BN);
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j * 32 + row_of(i, half) >= left) s[j][i] = -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[j][i]);
      top = fmaxf(top, __uint_as_float(lane_xor<32>(__float_as_uint(top))));
      const float next = fmaxf(m, top * c);
      if (__any(next > m)) {
        // (a row that has seen nothing has m -inf and nothing to scale)
        const float back = next > m ? __builtin_amdgcn_exp2f(m - next) : 1.0f;
        l *= back;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= back;
        m = next;
      }
      const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], c, -from));
          l += s[j][i];
        }
      // A value that is not finite must not reach the rows that do not see it:
      // zero times it is not zero.  Where a masked tile holds one, the finite
      // values are added as always and then the others key by key.
      bool bad = false;
      if (masked) {
#pragma unroll
        for (int j = 0; j < BN / 16; ++j)
#pragma unroll
          for (int d = 0; d < DT; ++d)
            bad |= any_not_finite<T>(read_columns<T, BN, DP>(v, j * 16, d * 32, lane));
      }
      if (__any(bad)) {
        const int left = (int)(seen.mine - base < BN ? seen.mine - base : BN);
#pragma unroll
        for (int j = 0; j < BN / 16; ++j) {
          const Operand<T> w = operand_of<T>(s[j >> 1], j & 1);
#pragma unroll
          for (int d = 0; d < DT; ++d)
            o[d] = multiply(finite_part<T>(read_columns<T, BN, DP>(v, j * 16, d * 32, lane)), w,
                            o[d]);
          for (int r = 0; r < 16; ++r) {
            const bool sees = j * 16 + r < left;
            const int slot = (r >> 3) * 4 + (r & 3);
            const bool own = (r >> 2 & 1) == half;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const Operand<T> a =
                  other_part<T>(read_columns<T, BN, DP>(v, j * 16, d * 32, lane), slot, own);
              if (!__any(any_not_finite<T>(a))) continue;
              const f32x16_t with = multiply(a, w, o[d]);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[d][i] = sees ? with[i] : o[d][i];
            }
          }
        }
        return;
      }
#pragma unroll
      for (int j = 0; j < BN / 16; ++j) {
        const Operand<T> w = operand_of<T>(s[j >> 1], j & 1);
#pragma unroll
        for (int d = 0; d < DT; ++d)
          o[d] = multiply(read_columns<T, BN, DP>(v, j * 16, d * 32, lane), w, o[d]);
      }
    };

    if (count > 0) fill(k0, v0, 0);
    for (int64_t n = 0; n < count; n += 2) {
      landed();
      if (n + 1 < count) fill(k1, v1, n + 1);
      work(k0, v0, n);
      if (n + 1 < count) {
        landed();
        if (n + 2 < count) fill(k0, v0, n + 2);
        work(k1, v1, n + 1);
      }
    }
    landed();  // nobody reads the tiles any more

    l += __uint_as_float(lane_xor<32>(__float_as_uint(l)));
    if (there) {
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int at = d * 32 + row_of(i, half);
          if (at < p.dim) {
            const f32x4_t w = {o[d][i] * inv, o[d][i + 1] * inv, o[d][i + 2] * inv,
                               o[d][i + 3] * inv};
            if constexpr (sizeof(S) == 4)
              *reinterpret_cast<f32x4_t *>(out + at) = w;
            else
              *reinterpret_cast<u32x2_u *>(out + at) =
                  u32x2_u{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3])};
          }
        }
      if (p.lse && half == 0)
        p.lse[row * p.heads + head] =
            l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) * kLn2 + logf(l);
    }
  }
}

template <typename T, int DP, int WAVES, int BN>
hipError_t run(const AttentionParams &p, hipStream_t stream) {
  const int64_t items = tile_count(p.tokens, p.batch, WAVES * 32) * p.heads;
  launch_kernel(attention_kernel<T, DP, WAVES, BN>, dim3(grid_of(items)), dim3(WAVES * kWave), 0,
                stream, p, items);
  return hipGetLastError();
}

template <typename T, int WAVES, int BN>
hipError_t by_dim(const AttentionParams &p, hipStream_t stream) {
  if (p.dim <= 32) return run<T, 32, WAVES, BN>(p, stream);
  if (p.dim <= 64) return run<T, 64, WAVES, BN>(p, stream);
  if (p.dim <= 96) return run<T, 96, WAVES, BN>(p, stream);
  return run<T, 128, WAVES, BN>(p, stream);
}

}  // namespace

hipError_t launch_attention(const AttentionParams &p, int dtype, hipStream_t stream) {
  // sequences of few rows take a wave each, and none waits for another
  const bool few = p.tokens / p.batch <= 48;
  if (dtype == kF32) return few ? by_dim<F32, 1, 32>(p, stream) : by_dim<F32, 4, 32>(p, stream);
  return few ? by_dim<BF16, 1, 32>(p, stream) : by_dim<BF16, 4, 64>(p, stream);
}

}  // namespace dlrm
