// attention_cached.hip -- attention of one query token for each sequence over a
// paged cache whose keys and values are held in 8 or 4 bits.
//
//   out[b, h] = sum_j softmax_j(scale q[b, h] . k[j]) v[j],   j < lengths[b]
//
// Bounded by the cache's bytes: every code is read once, for all heads that share
// its key head (16 of them at a time are the columns of 16 x 16 products; fewer
// leave columns idle, which costs matrix time that there is plenty of for bfloat16
// queries, but not for float32 ones).  A wave walks 64 keys a step.  Codes become
// bfloat16 (float32 for float32 queries) by the conversion instructions, which take
// the group's scale along and are exact; the weights are rounded to bfloat16 for
// bfloat16 queries.
//
// No value passes between lanes: in s^T = k q^T a lane holds a key's share of its
// dim, D/4 neighbouring elements (one load), the same ones of its head's query;
// the products' order of elements is free as long as both agree.  The
// exponentials of keys 4 g .. 4 g + 3 (g = lane / 16) of two blocks of 16 stay in
// the lane as eight slots of out^T += v^T p^T, for which the lane reads those
// eight tokens' values at D/16 neighbouring elements.
//
// Long sequences are split over workgroups, each sequence into equal shares of
// its own length; the shares' maxima, sums and outputs meet in a second kernel.
// (64 sequences of up to 8000 keys, 8 key heads of 128 in 8 bits, 32 bfloat16 heads: 120
// us, 5.0 TB/s; one of 131001 in 4 bits 31 us, 4.6 TB/s; their shares' meeting 5 us more
// each.  For float32 heads the two take 237 and 92 us for 127 and 36 in all.)
#include <math.h>

#include "attention_common.hpp"
#include "cache_common.hpp"

namespace dlrm {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 64;           // keys of a wave's step
constexpr int kHeads = 16;          // of a workgroup

__device__ __forceinline__ f32x4_t multiply16(const Operand<BF16> &a, const Operand<BF16> &b,
                                              f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v),
                                                 __builtin_bit_cast(bf16x8_t, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t multiply16(const Operand<F32> &a, const Operand<F32> &b,
                                              f32x4_t c) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e >> 2][e & 3], b.v[e >> 2][e & 3], c, 0, 0, 0);
  return c;
}

// Eight codes as an operand.
template <int BITS>
__device__ __forceinline__ void set_operand(Operand<BF16> &o, const Codes<BITS> &c, float unit) {
  o.v = u32x4_t{pair_bf16<0>(c, unit), pair_bf16<1>(c, unit), pair_bf16<2>(c, unit),
                pair_bf16<3>(c, unit)};
}
template <int BITS>
__device__ __forceinline__ void set_operand(Operand<F32> &o, const Codes<BITS> &c, float unit) {
  float v[8];
  values_of(c, unit, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) o.v[e >> 2][e & 3] = v[e];
}

// BYTES bytes from memory (1, 2, 4, 8, 16 or 32) as words.
template <int BYTES>
struct Words {
  static constexpr int N = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t w[N];
  __device__ __forceinline__ void load(const uint8_t *p) {
    if constexpr (BYTES == 1) {
      w[0] = *p;
    } else if constexpr (BYTES == 2) {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (BYTES == 8) {
      const uint64_t v = *reinterpret_cast<const uint64_t *>(p);
      w[0] = (uint32_t)v;
      w[1] = (uint32_t)(v >> 32);
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const u32x4_t v = reinterpret_cast<const u32x4_t *>(p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = v[e];
      }
    }
  }
};

// Eight tokens' codes at E neighbouring elements, as operands of E products:
// operand j holds element j of the eight tokens.
template <int E, int BITS, int N>
__device__ __forceinline__ void columns(const Words<N> (&v)[8], const float (&unit)[8],
                                        Operand<BF16> (&out)[E]) {
#pragma unroll
  for (int t = 0; t < 8; t += 2) {
    Codes<BITS> a{}, b{};
#pragma unroll
    for (int i = 0; i < Words<N>::N; ++i) {
      a.w[i] = v[t].w[i];
      b.w[i] = v[t + 1].w[i];
    }
    auto both = [&](int j, uint32_t x, uint32_t y) {   // (x0 x1) (y0 y1) -> (x0 y0) (x1 y1)
      out[j].v[t / 2] = __builtin_amdgcn_perm(y, x, 0x05040100);
      out[j + 1].v[t / 2] = __builtin_amdgcn_perm(y, x, 0x07060302);
    };
    both(0, pair_bf16<0>(a, unit[t]), pair_bf16<0>(b, unit[t + 1]));
    if constexpr (E > 2) both(2, pair_bf16<1>(a, unit[t]), pair_bf16<1>(b, unit[t + 1]));
    if constexpr (E > 4) {
      both(4, pair_bf16<2>(a, unit[t]), pair_bf16<2>(b, unit[t + 1]));
      both(6, pair_bf16<3>(a, unit[t]), pair_bf16<3>(b, unit[t + 1]));
    }
  }
}
template <int E, int BITS, int N>
__device__ __forceinline__ void columns(const Words<N> (&v)[8], const float (&unit)[8],
                                        Operand<F32> (&out)[E]) {
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    Codes<BITS> a{};
#pragma unroll
    for (int i = 0; i < Words<N>::N; ++i) a.w[i] = v[t].w[i];
    auto both = [&](int j, auto x) {
      out[j].v[t >> 2][t & 3] = x[0];
      out[j + 1].v[t >> 2][t & 3] = x[1];
    };
    both(0, pair_f32<0>(a, unit[t]));
    if constexpr (E > 2) both(2, pair_f32<1>(a, unit[t]));
    if constexpr (E > 4) {
      both(4, pair_f32<2>(a, unit[t]));
      both(6, pair_f32<3>(a, unit[t]));
    }
  }
}

// A share's result for one head: its sums relative to its maximum.
struct Share {
  float top, sum;
};

template <typename T, int D, int BITS>
__global__ __launch_bounds__(kWaves *kWave) void cached_kernel(CachedParams p, int splits,
                                                               int head_tiles, float *outs,
                                                               Share *shares, int64_t items) {
  using S = typename T::S;
  constexpr int STEPS = D / 32, E = D / 16, G = D / kGroup;
  constexpr int ROW = D * BITS / 8, KB = ROW / 4, VB = ROW / 16;
  constexpr int PITCH = D + 4;
  __shared__ float o_lds[kWaves][kHeads][PITCH];
  __shared__ Share s_lds[kWaves][kHeads];
  const int lane = threadIdx.x % kWave, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int page_bits = 31 - __builtin_clz(p.page);
  const float c = p.scale * kLog2e;
  const int kv_heads = p.heads / p.group;

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    // neighbouring workgroups take a sequence's key heads, whose pages lie together
    int64_t left = item;
    const int tile = (int)(left % head_tiles);
    left /= head_tiles;
    const int kv_head = (int)(left % kv_heads);
    left /= kv_heads;
    const int split = (int)(left % splits);
    const int64_t b = left / splits;
    const int group0 = tile * kHeads;
    const int heads = p.group - group0 < kHeads ? p.group - group0 : kHeads;
    const int64_t head0 = (int64_t)kv_head * p.group + group0;

    int64_t len = p.lengths[b];
    const int64_t most = p.max_pages << page_bits;
    len = len < 0 ? 0 : len > most ? most : len;
    const int64_t steps = (len + kStep - 1) / kStep;
    const int64_t first = steps * split / splits, last = steps * (split + 1) / splits;

    Operand<T> q[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      q[s] = zero_operand<T>();
      if (n < heads) {
        const S *at = (const S *)p.q.data + b * p.q.token + (head0 + n) * p.q.head + g * (D / 4) +
                      s * 8;
        if constexpr (sizeof(S) == 4) {
          q[s].v[0] = (f32x4_t) * reinterpret_cast<const f32x4_u *>(at);
          q[s].v[1] = (f32x4_t) * reinterpret_cast<const f32x4_u *>(at + 4);
        } else {
          q[s].v = (u32x4_t) * reinterpret_cast<const u32x4_u *>(at);
        }
      }
    }
    f32x4_t o[E];
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] = f32x4_t{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    for (int64_t step = first + wave; step < last; step += kWaves) {
      const int64_t key0 = step * kStep;
      // four blocks of 16 keys, each within a page
      Words<KB> kw[4];
      uint32_t ks[4][(STEPS + 3) / 4];
      Words<VB> vw[2][8];
      u32x4_t vs[4];   // scales of four tokens
      int there[4];    // keys of the block that are there
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t key = key0 + i * 16;
        int64_t page = key < len ? p.table[b * p.ld_table + (key >> page_bits)] : -1;
        there[i] = len - key < 16 ? (int)(len - key) : 16;
        if (page < 0 || page >= p.pages) there[i] = 0, page = 0;
        const int64_t row = (page * kv_heads + kv_head) * p.page + (key & (p.page - 1));
        kw[i].load(p.k_codes + (row + n) * ROW + g * KB);
        const uint8_t *sc = p.k_scales + (row + n) * G;
        ks[i][0] = G == 4 ? sc[g] : G == 2 ? sc[g >> 1] : sc[0];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vw[i >> 1][(i & 1) * 4 + e].load(p.v_codes + (row + g * 4 + e) * ROW + n * VB);
        const uint8_t *vsc = p.v_scales + (row + g * 4) * G;
        if constexpr (G == 4) {
          vs[i] = *reinterpret_cast<const u32x4_t *>(vsc);
        } else if constexpr (G == 2) {
          const u32x2_u w = *reinterpret_cast<const u32x2_u *>(vsc);
          vs[i] = u32x4_t{w[0] & 0xffff, w[0] >> 16, w[1] & 0xffff, w[1] >> 16};
        } else {
          const uint32_t w = *reinterpret_cast<const uint32_t *>(vsc);
          vs[i] = u32x4_t{w & 0xff, w >> 8 & 0xff, w >> 16 & 0xff, w >> 24};
        }
      }
      const bool whole = there[0] == 16 && there[1] == 16 && there[2] == 16 && there[3] == 16;
      f32x4_t s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = f32x4_t{0, 0, 0, 0};
        const float unit = unit_of(ks[i][0]);
#pragma unroll
        for (int e = 0; e < STEPS; ++e) {
          Codes<BITS> codes;
#pragma unroll
          for (int w = 0; w < BITS / 4; ++w) codes.w[w] = kw[i].w[e * (BITS / 4) + w];
          Operand<T> k;
          set_operand(k, codes, unit);
          s[i] = multiply16(k, q[e], s[i]);
        }
      }
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (g * 4 + e >= there[i]) {
              s[i][e] = -INFINITY;
              vs[i][e] = 0x7f7f7f7f;
#pragma unroll
              for (int w = 0; w < Words<VB>::N; ++w) vw[i >> 1][(i & 1) * 4 + e].w[w] = 0;
            }
      }
      float top = s[0][0];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i][e]);
      top = fmaxf(top, __uint_as_float(lane_xor<16>(__float_as_uint(top))));
      top = fmaxf(top, __uint_as_float(lane_xor<32>(__float_as_uint(top))));
      const float next = fmaxf(m, top * c);
      if (__any(next > m)) {
        const float back = next > m ? __builtin_amdgcn_exp2f(m - next) : 1.0f;
        l *= back;
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] *= back;
        m = next;
      }
      const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float w[8], unit[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = 2 * h + (e >> 2);
          w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][e & 3], c, -from));
          l += w[e];
          const uint32_t sc = vs[i][e & 3];
          unit[e] = unit_of(sc >> (n * E / kGroup * 8) & 0xff);
        }
        Operand<T> pw;
        if constexpr (sizeof(S) == 4) {
#pragma unroll
          for (int e = 0; e < 8; ++e) pw.v[e >> 2][e & 3] = w[e];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) pw.v[e] = pack_bf16(w[2 * e], w[2 * e + 1]);
        }
        Operand<T> v[E];
        columns<E, BITS>(vw[h], unit, v);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = multiply16(v[j], pw, o[j]);
      }
    }
    l += __uint_as_float(lane_xor<16>(__float_as_uint(l)));
    l += __uint_as_float(lane_xor<32>(__float_as_uint(l)));
    // output i of product j is element (4 g + i) E + j of head n
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) o_lds[wave][n][(g * 4 + i) * E + j] = o[j][i];
    if (g == 0) s_lds[wave][n] = Share{m, l};
    __syncthreads();
    for (int i = threadIdx.x; i < heads * D; i += kWaves * kWave) {
      const int h = i / D, d = i % D;
      float top = -INFINITY, sum = 0.0f, out = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_lds[w][h].top);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = s_lds[w][h].top == -INFINITY
                            ? (s_lds[w][h].sum != 0.0f ? 1.0f : 0.0f)   // (a NaN is kept)
                            : __builtin_amdgcn_exp2f(s_lds[w][h].top - top);
        sum = __builtin_fmaf(s_lds[w][h].sum, f, sum);
        out = __builtin_fmaf(o_lds[w][h][d], f, out);
      }
      if (splits == 1) {
        S *at = (S *)p.out.data + b * p.out.token + (head0 + h) * p.out.head + d;
        store1<T>(at, sum == 0.0f ? 0.0f : out / sum);
      } else {
        const int64_t at = (b * p.heads + head0 + h) * splits + split;
        outs[at * D + d] = out;
        if (d == 0) shares[at] = Share{top, sum};
      }
    }
    __syncthreads();
  }
}

// The shares of a head: 32 of its elements by GROUPS groups of lanes, each an
// equal part of the shares.  Few shares take one group (64 sequences of 32 heads,
// 4 shares: 5 us, with eight groups 10), many take eight (one sequence, 128
// shares: 7 us, with one group 45).
constexpr int kJoinThreads = 256;
template <typename T, int D, int GROUPS>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(CachedParams p, int splits,
                                                            const float *outs, const Share *shares,
                                                            int64_t items) {
  using S = typename T::S;
  constexpr int EACH = kJoinThreads / 32 / GROUPS;   // items of a workgroup
  __shared__ float parts[GROUPS][32], sums[GROUPS];
  const int e = threadIdx.x & 31, g = threadIdx.x / 32 % GROUPS;
  for (int64_t item0 = (int64_t)blockIdx.x * EACH; item0 < items;
       item0 += (int64_t)gridDim.x * EACH) {
    int64_t item = item0 + threadIdx.x / 32 / GROUPS;
    const bool there = item < items;
    item = there ? item : items - 1;
    const int64_t row = item / (D / 32);
    const int d = (int)(item % (D / 32)) * 32 + e;
    const Share *s = shares + row * splits;
    float top = -INFINITY;
    for (int i = e; i < splits; i += 32) top = fmaxf(top, s[i].top);
#pragma unroll
    for (int x = 1; x < 32; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
    float sum = 0.0f, out = 0.0f;
#pragma unroll 4
    for (int i = g; i < splits; i += GROUPS) {
      const float f = s[i].top == -INFINITY ? (s[i].sum != 0.0f ? 1.0f : 0.0f)
                                            : __builtin_amdgcn_exp2f(s[i].top - top);
      sum = __builtin_fmaf(s[i].sum, f, sum);
      out = __builtin_fmaf(outs[(row * splits + i) * D + d], f, out);
    }
    if constexpr (GROUPS > 1) {
      parts[g][e] = out;
      if (e == 0) sums[g] = sum;
      __syncthreads();
      sum = out = 0.0f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) {
        sum += sums[i];
        out += parts[i][e];
      }
      __syncthreads();
    }
    if (there && g == 0) {
      const int64_t b = row / p.heads, h = row - b * p.heads;
      store1<T>((S *)p.out.data + b * p.out.token + h * p.out.head + d,
                sum == 0.0f ? 0.0f : out / sum);
    }
  }
}

int head_tiles_of(int group) { return (group + kHeads - 1) / kHeads; }

// Shares of a sequence: two workgroups a CU (one sequence of 131001 keys, 8 key heads
// of 128 in 4 bits: 64 shares 35 us, 32 43, 128 42), or where sequences are many,
// four shares each, since the long ones among them would end last; no more than its
// row of the table has steps for.  A sequence shorter than that row leaves shares
// empty (64 of 50 keys take 26 us under rows of 1024 keys as of 131072).
int splits_of(int64_t batch, int heads, int kv_heads, int64_t max_pages, int page) {
  const int64_t groups = batch * kv_heads * head_tiles_of(heads / kv_heads);
  const int64_t most = (max_pages * page + kWaves * kStep - 1) / (kWaves * kStep);
  int64_t want = (512 + groups - 1) / groups;
  want = want < 4 ? 4 : want > 256 ? 256 : want;
  want = want < most ? want : most;
  return want < 1 ? 1 : (int)want;
}

template <typename T, int D, int BITS>
hipError_t run(const CachedParams &p, void *ws, hipStream_t stream) {
  const int kv_heads = p.heads / p.group, tiles = head_tiles_of(p.group);
  const int splits = splits_of(p.batch, p.heads, kv_heads, p.max_pages, p.page);
  const int64_t items = p.batch * kv_heads * tiles * splits, rows = p.batch * p.heads;
  float *outs = (float *)ws;
  Share *shares = (Share *)(outs + rows * splits * D);
  launch_kernel(cached_kernel<T, D, BITS>, dim3(grid_of(items)), dim3(kWaves * kWave), 0, stream,
                p, splits, tiles, outs, shares, items);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t pieces = rows * (D / 32);
  if (splits <= 16)
    launch_kernel(join_kernel<T, D, 1>, dim3(grid_of((pieces + 7) / 8)), dim3(kJoinThreads), 0,
                  stream, p, splits, (const float *)outs, (const Share *)shares, pieces);
  else
    launch_kernel(join_kernel<T, D, 8>, dim3(grid_of(pieces)), dim3(kJoinThreads), 0, stream, p,
                  splits, (const float *)outs, (const Share *)shares, pieces);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t by_bits(const CachedParams &p, int bits, void *ws, hipStream_t stream) {
  return bits == 8 ? run<T, D, 8>(p, ws, stream) : run<T, D, 4>(p, ws, stream);
}
template <typename T>
hipError_t by_dim(const CachedParams &p, int dim, int bits, void *ws, hipStream_t stream) {
  if (dim == 32) return by_bits<T, 32>(p, bits, ws, stream);
  if (dim == 64) return by_bits<T, 64>(p, bits, ws, stream);
  return by_bits<T, 128>(p, bits, ws, stream);
}

}  // namespace

size_t cached_workspace(int64_t batch, int heads, int kv_heads, int dim, int64_t max_pages,
                        int page) {
  const int splits = splits_of(batch, heads, kv_heads, max_pages, page);
  return splits == 1 ? 0 : (size_t)batch * heads * splits * (dim * sizeof(float) + sizeof(Share));
}

hipError_t launch_cached(const CachedParams &p, int dtype, int dim, int bits, void *ws,
                         hipStream_t stream) {
  return dtype == kF32 ? by_dim<F32>(p, dim, bits, ws, stream)
                       : by_dim<BF16>(p, dim, bits, ws, stream);
}

}  // namespace dlrm
