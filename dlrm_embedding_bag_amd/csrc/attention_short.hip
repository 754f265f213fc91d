// attention_short.hip -- attention over packed sequences of few rows, and its
// gradient: the formulas of attention_packed.hip and attention_grad.hip, by waves
// that each hold 16 rows (or keys) of one head and walk the others 16 at a time.
//
// Histories of some ten rows fill a quarter of a tile of 32 x 32 scores, but most of
// one of 16 x 16, and their rows are read once or twice each, so nothing goes through
// LDS: a lane reads its part of the rows from memory in just the layouts that the
// products take.  A wave waits for memory more than it computes, and two to four of a
// SIMD cover each other.  (2048 sequences of up to 20 rows, 4 heads of 64 in float32:
// 24 us, 3.5 TB/s of what must be read and written, where tiles of 32 took 45; the
// gradient 83 us for 120.  One kernel for all of the gradient, which reads the rows of
// short sequences once, leaves registers for fewer waves: of 8 heads it took 128 us
// for 134, but of 128 elements in bfloat16 211 for 169.)
#include <math.h>

#include "attention_forward.hpp"

namespace dlrm {
namespace {

// The product of 16 x 16 outputs, out[m][n] += sum over 16 k of a[m][k] b[n][k].
// Lane r + 16 g holds slots 4 g .. 4 g + 3 of the contraction, in any order that a
// and b share, of row r of a and of row r of b; of the outputs it holds column r and
// rows 4 g + i, which makes them the operand of a product over those rows.
template <typename T>
struct Quad;
template <>
struct Quad<BF16> {
  u32x2_t v;
};
template <>
struct Quad<F32> {
  f32x4_t v;
};
__device__ __forceinline__ f32x4_t multiply(const Quad<BF16> &a, const Quad<BF16> &b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(i16x4_t, a.v),
                                                   __builtin_bit_cast(i16x4_t, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t multiply(const Quad<F32> &a, const Quad<F32> &b, f32x4_t c) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
  return c;
}
template <typename T>
__device__ __forceinline__ Quad<T> quad_of(const f32x4_t &c) {
  Quad<T> o;
  if constexpr (sizeof(typename T::S) == 4)
    o.v = c;
  else
    o.v = u32x2_t{pack_bf16(c[0], c[1]), pack_bf16(c[2], c[3])};
  return o;
}

__device__ __forceinline__ float dot(const Quad<BF16> &a, const Quad<BF16> &b, float sum) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sum = __builtin_fmaf(bf16_lo(a.v[e]), bf16_lo(b.v[e]), sum);
    sum = __builtin_fmaf(bf16_hi(a.v[e]), bf16_hi(b.v[e]), sum);
  }
  return sum;
}
__device__ __forceinline__ float dot(const Quad<F32> &a, const Quad<F32> &b, float sum) {
#pragma unroll
  for (int e = 0; e < 4; ++e) sum = __builtin_fmaf(a.v[e], b.v[e], sum);
  return sum;
}

__device__ __forceinline__ uint32_t load4_from(__amdgpu_buffer_rsrc_t b, uint32_t from) {
  return __builtin_amdgcn_raw_buffer_load_b32(b, from, 0, 0);
}
__device__ __forceinline__ u32x2_t load8_from(__amdgpu_buffer_rsrc_t b, uint32_t from) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(b, from, 0, 0));
}
__device__ __forceinline__ float add_quarters(float v) {
  v += __uint_as_float(lane_xor<16>(__float_as_uint(v)));
  return v + __uint_as_float(lane_xor<32>(__float_as_uint(v)));
}
__device__ __forceinline__ float max_quarters(float v) {
  v = fmaxf(v, __uint_as_float(lane_xor<16>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(lane_xor<32>(__float_as_uint(v))));
}

// Up to 16 rows of a tensor in memory, `left` of them there; what lies behind them
// or behind a row's end reads as zeros and is not stored.
template <typename T, int DP>
struct Rows {
  using S = typename T::S;
  static constexpr uint32_t E = sizeof(S);
  static constexpr int STEPS = DP / 16;            // quads of a row
  // columns: lane r holds W neighbouring ones of each of CHUNKS, from W r on
  static constexpr int W = DP % 64 ? 2 : 4, CHUNKS = DP / (16 * W);
  __amdgpu_buffer_rsrc_t buffer;
  uint32_t row;   // bytes
  int left, dim;
  __device__ __forceinline__ Rows(const void *base, int64_t stride, int left_, int dim_)
      : buffer(buffer_of(base, ((uint32_t)(left_ < 16 ? left_ - 1 : 15) * (uint32_t)stride + dim_) * E)),
        row((uint32_t)stride * E), left(left_), dim(dim_) {}

  // Row r, for products over its elements.
  __device__ __forceinline__ void load(Quad<T> (&q)[STEPS], int r, int g) const {
    const uint32_t at = (uint32_t)r * row;
    if constexpr (E == 4) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int c = s * 16 + g * 4;
        q[s].v = __builtin_bit_cast(
            f32x4_t, load_from(buffer, r < left && c < dim ? at + c * E : kNowhere));
      }
    } else {
#pragma unroll
      for (int s = 0; s < STEPS; s += 2) {
        const int c = s * 16 + g * 8;
        const u32x4_t w = load_from(buffer, r < left && c < dim ? at + c * E : kNowhere);
        q[s].v = u32x2_t{w[0], w[1]};
        q[s + 1].v = u32x2_t{w[2], w[3]};
      }
    }
  }

  // Rows 4 g .. 4 g + 3, the lane's columns, for products over rows.
  struct Columns {
    uint32_t v[CHUNKS][4][W * E / 4];
    __device__ __forceinline__ Quad<T> quad(int chunk, int t) const {
      Quad<T> o;
      if constexpr (E == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o.v[e] = __uint_as_float(v[chunk][e][t]);
      } else {
        const uint32_t pick = t & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          o.v[e] = __builtin_amdgcn_perm(v[chunk][2 * e + 1][t / 2], v[chunk][2 * e][t / 2], pick);
      }
      return o;
    }
  };
  __device__ __forceinline__ void load(Columns &q, int r, int g) const {
#pragma unroll
    for (int h = 0; h < CHUNKS; ++h) {
      const int c = h * 16 * W + r * W;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = g * 4 + e;
        const uint32_t at = k < left && c < dim ? (uint32_t)k * row + c * E : kNowhere;
        uint32_t(&to)[W * E / 4] = q.v[h][e];
        if constexpr (W * E == 16) {
          const u32x4_t w = load_from(buffer, at);
#pragma unroll
          for (int i = 0; i < 4; ++i) to[i] = w[i];
        } else if constexpr (W * E == 8) {
          const u32x2_t w = load8_from(buffer, at);
          to[0] = w[0];
          to[1] = w[1];
        } else {
          to[0] = load4_from(buffer, at);
        }
      }
    }
  }

  // What products of columns leave a lane of row r: 4 W elements of each chunk.
  using Sums = f32x4_t[CHUNKS][W];
  __device__ __forceinline__ static float of(const Sums &o, int h, int i) {
    return o[h][i % W][i / W];
  }
  __device__ __forceinline__ void store(const Sums &o, float scale, int r, int g) const {
    constexpr int N = 16 / E;
#pragma unroll
    for (int h = 0; h < CHUNKS; ++h)
#pragma unroll
      for (int i = 0; i < 4 * W; i += N) {
        const int c = h * 16 * W + g * 4 * W + i;
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = E == 4 ? __float_as_uint(of(o, h, i + e) * scale)
                        : pack_bf16(of(o, h, i + 2 * e % N) * scale,
                                    of(o, h, i + (2 * e + 1) % N) * scale);
        store_to(buffer, r < left && c < dim ? (uint32_t)r * row + c * E : kNowhere, w);
      }
  }
};
template <typename T, int DP>
__device__ __forceinline__ void add_products(typename Rows<T, DP>::Sums &o,
                                             const typename Rows<T, DP>::Columns &a,
                                             const Quad<T> &b) {
#pragma unroll
  for (int h = 0; h < Rows<T, DP>::CHUNKS; ++h)
#pragma unroll
    for (int t = 0; t < Rows<T, DP>::W; ++t) o[h][t] = multiply(a.quad(h, t), b, o[h][t]);
}

template <typename T, int DP>
__device__ __forceinline__ void clear(typename Rows<T, DP>::Sums &o) {
#pragma unroll
  for (int h = 0; h < Rows<T, DP>::CHUNKS; ++h)
#pragma unroll
    for (int t = 0; t < Rows<T, DP>::W; ++t) o[h][t] = f32x4_t{};
}

// (Left to itself the compiler asks for all rows at once and takes the registers of a
// second or fourth wave: of 2048 sequences of about 10 rows, 8 heads of 64 in float32
// 49 us, 42 so; of 128 193 and 159.  The gradient's kernels lose by any such bound.)
template <typename T, int DP>
__global__ __launch_bounds__(kWave, (sizeof(typename T::S) == 4 && DP > 64 ? 3 : 4))
void attention_short_kernel(AttentionParams p, int64_t items) {
  using S = typename T::S;
  using R = Rows<T, DP>;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const float c = p.scale * kLog2e;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int dim = in_loop(p.dim);
    const Item at = item_of(item, tile_count(p.tokens, p.batch, 16), p.heads);
    const int head = at.head;
    const Tile t = find_tile(p.offsets, p.batch, p.tokens, at.tile, 16);
    if (t.left <= 0) continue;
    if (t.sequence < 0) {
      if (r < t.left && g == 0) put_nothing<T>(p, (int64_t)t.row + r, head);
      continue;
    }
    const Range keys = p.kv_offsets ? rows_of(p.kv_offsets, p.batch, p.kv_tokens, t.sequence)
                                    : Range{t.first, t.row - t.first + t.left};
    const SeenKeys seen(p.causal, keys.count, t.left, 16, 0, 16);
    const int seen_keys = seen.by(r), kv_head = head / p.group;
    const S *kbase = (const S *)p.k.data + keys.first * p.k.token + kv_head * p.k.head;
    const S *vbase = (const S *)p.v.data + keys.first * p.v.token + kv_head * p.v.head;
    Quad<T> q[R::STEPS];
    R((const S *)p.q.data + t.row * p.q.token + head * p.q.head, p.q.token, t.left, dim).load(q, r, g);
    typename R::Sums o;
    clear<T, DP>(o);
    float m = -INFINITY, l = 0.0f;
    int loose = -1;   // the first key whose values are not all added

    for (int base = 0; base < seen.wave_any; base += 16) {
      Quad<T> k[R::STEPS];
      typename R::Columns v;
      R(kbase + base * p.k.token, p.k.token, keys.count - base, dim).load(k, r, g);
      R(vbase + base * p.v.token, p.v.token, keys.count - base, dim).load(v, r, g);
      f32x4_t s = {};
#pragma unroll
      for (int i = 0; i < R::STEPS; ++i) s = multiply(k[i], q[i], s);
      if (seen.wave_all - base < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (base + g * 4 + i >= seen_keys) s[i] = -INFINITY;
        // a value that is not finite must not reach the rows that do not see it, and
        // zero times it is not zero: it is left out here and added at the end
        if (p.causal) {
          uint32_t others = 0;
#pragma unroll
          for (int h = 0; h < R::CHUNKS; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int i = 0; i < (int)(R::W * R::E / 4); ++i) others |= not_finite<T>(v.v[h][e][i]);
          if (__any(others != 0)) {
            loose = loose < 0 ? base : loose;
#pragma unroll
            for (int h = 0; h < R::CHUNKS; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < (int)(R::W * R::E / 4); ++i) v.v[h][e][i] = finite<T>(v.v[h][e][i]);
          }
        }
      }
      const float top = max_quarters(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])));
      const float next = fmaxf(m, top * c);
      if (__any(next > m + kSlack)) {
        const bool mine = next > m + kSlack;
        const float back = mine ? __builtin_amdgcn_exp2f(m - next) : 1.0f;
        l *= back;
#pragma unroll
        for (int h = 0; h < R::CHUNKS; ++h)
#pragma unroll
          for (int d = 0; d < R::W; ++d) o[h][d] *= back;
        m = mine ? next : m;
      }
      const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -from));
        l += s[i];
      }
      add_products<T, DP>(o, v, quad_of<T>(s));
    }

    if (loose >= 0)
      for (int j = loose; j < seen_keys; ++j)
#pragma unroll
        for (int h = 0; h < R::CHUNKS; ++h)
#pragma unroll
          for (int i = 0; i < 4 * R::W; ++i) {
            const int d = h * 16 * R::W + g * 4 * R::W + i;
            const float x = d < dim ? load1<T>(vbase + (int64_t)j * p.v.token + d) : 0.0f;
            if ((__float_as_uint(x) & kInfinity) == kInfinity) o[h][i % R::W][i / R::W] += x;
          }
    l = add_quarters(l);
    R((S *)p.out.data + t.row * p.out.token + head * p.out.head, p.out.token, t.left, dim)
        .store(o, l > 0.0f || l != l ? 1.0f / l : 0.0f, r, g);
    if (p.lse && g == 0 && r < t.left) p.lse[((int64_t)t.row + r) * p.heads + head] = lse_of(m, l);
  }
}

// Rows: dq, and the rows' statistics.
template <typename T, int DP>
__global__ __launch_bounds__(kWave) void grad_short_rows_kernel(AttentionGradParams p, float *ws,
                                                                int64_t items) {
  using S = typename T::S;
  using R = Rows<T, DP>;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const float c = p.scale * kLog2e;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int dim = in_loop(p.dim);
    const Item at = item_of(item, tile_count(p.tokens, p.batch, 16), p.heads);
    const int head = at.head;
    const Tile t = find_tile(p.offsets, p.batch, p.tokens, at.tile, 16);
    if (t.left <= 0) continue;
    const int64_t row = (int64_t)t.row + r;
    const bool there = r < t.left;
    if (t.sequence < 0) {
      if (there && g == 0 && p.fill & 1) {
        S *dq = (S *)p.dq.data + row * p.dq.token + head * p.dq.head;
        for (int d = 0; d < dim; ++d) dq[d] = 0;
      }
      continue;
    }
    const Range keys = p.kv_offsets ? rows_of(p.kv_offsets, p.batch, p.kv_tokens, t.sequence)
                                    : Range{t.first, t.row - t.first + t.left};
    const SeenKeys seen(p.causal, keys.count, t.left, 16, 0, 16);
    const int seen_keys = seen.by(r), kv_head = head / p.group;
    const S *kbase = (const S *)p.k.data + keys.first * p.k.token + kv_head * p.k.head;
    const S *vbase = (const S *)p.v.data + keys.first * p.v.token + kv_head * p.v.head;
    Quad<T> q[R::STEPS], gr[R::STEPS];
    float delta = 0.0f;
    R((const S *)p.q.data + t.row * p.q.token + head * p.q.head, p.q.token, t.left, dim).load(q, r, g);
    R((const S *)p.grad.data + t.row * p.grad.token + head * p.grad.head, p.grad.token, t.left, dim)
        .load(gr, r, g);
    {
      Quad<T> o[R::STEPS];
      R((const S *)p.out.data + t.row * p.out.token + head * p.out.head, p.out.token, t.left, dim)
          .load(o, r, g);
#pragma unroll
      for (int i = 0; i < R::STEPS; ++i) delta = dot(gr[i], o[i], delta);
    }
    delta = add_quarters(delta);
    float lse2 = there ? p.lse[row * p.heads + head] * kLog2e : INFINITY;
    if (lse2 == -INFINITY) lse2 = INFINITY;
    if (there && g == 0) {
      const Stats stats(ws, p.tokens, p.heads);
      stats.turned_lse2[head * p.tokens + row] = turned(lse2);
      stats.minus_delta[head * p.tokens + row] = -delta;
    }
    typename R::Sums o;
    clear<T, DP>(o);
    for (int base = 0; base < seen.wave_any; base += 16) {
      Quad<T> k[R::STEPS], v[R::STEPS];
      typename R::Columns kc;
      const R kr(kbase + base * p.k.token, p.k.token, keys.count - base, dim);
      kr.load(k, r, g);
      R(vbase + base * p.v.token, p.v.token, keys.count - base, dim).load(v, r, g);
      kr.load(kc, r, g);
      f32x4_t s = {}, dp = {};
#pragma unroll
      for (int i = 0; i < R::STEPS; ++i) {
        s = multiply(k[i], q[i], s);
        dp = multiply(v[i], gr[i], dp);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse2)) * (dp[i] - delta);
        if (base + g * 4 + i >= seen_keys) s[i] = 0.0f;
      }
      add_products<T, DP>(o, kc, quad_of<T>(s));
    }
    R((S *)p.dq.data + t.row * p.dq.token + head * p.dq.head, p.dq.token, t.left, dim)
        .store(o, p.scale, r, g);
  }
}

// Keys: dk and dv.  A lane holds one of its wave's 16.
template <typename T, int DP>
__global__ __launch_bounds__(kWave) void grad_short_keys_kernel(AttentionGradParams p, float *ws,
                                                                int kv_heads, int64_t items) {
  using S = typename T::S;
  using R = Rows<T, DP>;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const float c = p.scale * kLog2e;
  const int32_t *key_offsets = p.kv_offsets ? p.kv_offsets : p.offsets;
  const Stats stats(ws, p.tokens, p.heads);
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int dim = in_loop(p.dim);
    const int64_t tiles = tile_count(p.kv_tokens, p.batch, 16);
    const Item at = item_of(item, tiles, kv_heads);
    const int kv_head = at.head;
    const Tile t = find_tile(key_offsets, p.batch, p.kv_tokens, tiles - 1 - at.tile, 16);
    if (t.left <= 0) continue;
    if (t.sequence < 0) {
      if (r < t.left && g == 0) {
        const int64_t key = (int64_t)t.row + r;
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
    // the first row that sees the key: as far from the last row as it from the last key
    auto first_row = [&](int key) {
      const int f = p.causal ? rows.count - (t.left - key) : 0;
      return f < 0 ? 0 : f;
    };
    const int from_row = r < t.left ? first_row(r) : rows.count;
    Quad<T> k[R::STEPS], v[R::STEPS];
    R((const S *)p.k.data + t.row * p.k.token + kv_head * p.k.head, p.k.token, t.left, dim)
        .load(k, r, g);
    R((const S *)p.v.data + t.row * p.v.token + kv_head * p.v.head, p.v.token, t.left, dim)
        .load(v, r, g);
    typename R::Sums ok, ov;
    clear<T, DP>(ok);
    clear<T, DP>(ov);
    for (int j = 0; j < p.group; ++j) {
      const int64_t head = (int64_t)kv_head * p.group + j;
      for (int base = first_row(0) & ~15; base < rows.count; base += 16) {
        const int64_t row = (int64_t)rows.first + base;
        const int left = rows.count - base, n = (left < 16 ? left : 16) * 4;
        const R qr((const S *)p.q.data + row * p.q.token + head * p.q.head, p.q.token, left, dim);
        const R gr((const S *)p.grad.data + row * p.grad.token + head * p.grad.head, p.grad.token,
                   left, dim);
        const auto lse_at = buffer_of(stats.turned_lse2 + head * p.tokens + row, n);
        const auto delta_at = buffer_of(stats.minus_delta + head * p.tokens + row, n);
        Quad<T> a[R::STEPS];
        typename R::Columns ac;
        float lse2[4];
        f32x4_t s = {}, dp;
        qr.load(a, r, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lse2[i] = turned(__uint_as_float(load4_from(lse_at, (g * 4 + i) * 4)));
          dp[i] = __uint_as_float(load4_from(delta_at, (g * 4 + i) * 4));
        }
        gr.load(ac, r, g);
#pragma unroll
        for (int i = 0; i < R::STEPS; ++i) s = multiply(a[i], k[i], s);
        gr.load(a, r, g);
#pragma unroll
        for (int i = 0; i < R::STEPS; ++i) dp = multiply(a[i], v[i], dp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse2[i]));
          dp[i] *= s[i];
          if (base + g * 4 + i < from_row) s[i] = dp[i] = 0.0f;
        }
        add_products<T, DP>(ov, ac, quad_of<T>(s));
        qr.load(ac, r, g);
        add_products<T, DP>(ok, ac, quad_of<T>(dp));
      }
    }
    R((S *)p.dk.data + t.row * p.dk.token + kv_head * p.dk.head, p.dk.token, t.left, dim)
        .store(ok, p.scale, r, g);
    R((S *)p.dv.data + t.row * p.dv.token + kv_head * p.dv.head, p.dv.token, t.left, dim)
        .store(ov, 1.0f, r, g);
  }
}

template <typename T, int DP>
hipError_t run(const AttentionParams &p, hipStream_t stream) {
  const int64_t items = tile_count(p.tokens, p.batch, 16) * p.heads;
  launch_kernel(attention_short_kernel<T, DP>, dim3(grid_of(items)), dim3(kWave), 0, stream, p, items);
  return hipGetLastError();
}
template <typename T, int DP>
hipError_t run(const AttentionGradParams &p, float *ws, hipStream_t stream) {
  if (p.tokens) {
    const int64_t items = tile_count(p.tokens, p.batch, 16) * p.heads;
    launch_kernel(grad_short_rows_kernel<T, DP>, dim3(grid_of(items)), dim3(kWave), 0, stream, p, ws,
                  items);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p.kv_tokens) return hipSuccess;
  const int kv_heads = p.heads / p.group;
  const int64_t items = tile_count(p.kv_tokens, p.batch, 16) * kv_heads;
  launch_kernel(grad_short_keys_kernel<T, DP>, dim3(grid_of(items)), dim3(kWave), 0, stream, p, ws,
                kv_heads, items);
  return hipGetLastError();
}

template <typename T, typename P, typename... A>
hipError_t by_dim(const P &p, A... a) {
  if (p.dim <= 32) return run<T, 32>(p, a...);
  if (p.dim <= 64) return run<T, 64>(p, a...);
  if (p.dim <= 96) return run<T, 96>(p, a...);
  return run<T, 128>(p, a...);
}

}  // namespace

hipError_t launch_attention_short(const AttentionParams &p, int dtype, hipStream_t stream) {
  return dtype == kF32 ? by_dim<F32>(p, stream) : by_dim<BF16>(p, stream);
}

hipError_t launch_attention_grad_short(const AttentionGradParams &p, int dtype, void *workspace,
                                       hipStream_t stream) {
  float *ws = (float *)workspace;
  return dtype == kF32 ? by_dim<F32>(p, ws, stream) : by_dim<BF16>(p, ws, stream);
}

}  // namespace dlrm
