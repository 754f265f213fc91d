// qk_norm_rope.hip -- RMS norm of the query and key heads with the rotation by
// position in the same pass, and its gradient.
//
// For a head's row x of n elements, with weight w, position t and frequencies f:
//   u = x / sqrt(mean(x^2) + eps)        v = u w
//   (a, b) of v's pair i  ->  (a cos(t f_i) - b sin(t f_i), a sin(t f_i) + b cos(t f_i))
// Pairs are elements (i, i + pairs), or (2i, 2i + 1) if interleaved; elements
// from 2 pairs on are not turned.  With the gradient dy turned back to dv:
//   dw = sum over rows of dv u           g = dv w
//   dx = (g - u mean(g u)) / sqrt(mean(x^2) + eps)
//
// Bounded by memory: every row is read and written once.  A workgroup takes a
// few tokens: its threads first make the tokens' cosines and sines, one pair a
// thread, and leave them in LDS, where all heads of a token find them.  Then
// every group of lanes takes a row, each lane both members of its pairs, so a
// row never leaves its lanes' registers.  (16384 tokens of 40 heads of 128 in
// bfloat16: 69 us, 4.8 TB/s; the gradient of 8191 of 20 of 96 in float32 51 us.)
#include <math.h>

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = kMaxRopeDim / 2;

// cos and sin of position * frequency.  The angle and its reduction to an
// eighth of a turn are in 64 bits: far positions leave it thousands of turns.
__device__ __forceinline__ float2 turn_of(int position, float freq) {
  const double turns = (double)position * (double)freq * 0.15915494309189533577;
  const double part = turns - rint(turns);
  const double quarter = rint(part * 4.0);
  float s, c;
  sincospif((float)((part - quarter * 0.25) * 2.0), &s, &c);
  const int n = (int)quarter & 3;
  const float cs = n & 1 ? s : c, sn = n & 1 ? c : s;
  return make_float2(n == 1 || n == 2 ? -cs : cs, n >= 2 ? -sn : sn);
}

// What a lane holds of its row: N elements from `lo` and N from `hi`.
template <int N>
struct Slot {
  int lo, hi, pair;  // pair: of the first element
  bool there, turned;
};

template <int N, bool INTER>
__device__ __forceinline__ Slot<N> slot_of(int c, int dim, int pairs) {
  Slot<N> s;
  s.there = c < dim / (2 * N);
  s.pair = c * N;
  s.turned = s.pair < pairs;
  if (INTER || !s.turned) {
    s.lo = 2 * N * c;
    s.hi = s.lo + N;
  } else {
    s.lo = s.pair;
    s.hi = pairs + s.pair;
  }
  return s;
}

template <typename T, int N>
__device__ __forceinline__ void load_slot(const typename T::S *row, const Slot<N> &s,
                                          float (&v)[2 * N]) {
  float a[N], b[N];
  if constexpr (N == 8) {
    load8<T>(row + s.lo, a);
    load8<T>(row + s.hi, b);
  } else {
    load4<T>(row + s.lo, a);
    load4<T>(row + s.hi, b);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    v[e] = a[e];
    v[N + e] = b[e];
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_slot(typename T::S *row, const Slot<N> &s,
                                           const float (&v)[2 * N]) {
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    typename T::S *p = row + (part ? s.hi : s.lo);
    const float *a = v + part * N;
    if constexpr (sizeof(typename T::S) == 4) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        f32x4_u w = {a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]};
        *reinterpret_cast<f32x4_u *>(p + 4 * i) = w;
      }
    } else if constexpr (N == 8) {
      u32x4_u w = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]),
                   pack_bf16(a[6], a[7])};
      *reinterpret_cast<u32x4_u *>(p) = w;
    } else {
      u32x2_u w = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
      *reinterpret_cast<u32x2_u *>(p) = w;
    }
  }
}

// The two members of pair e in a slot's elements.
template <int N, bool INTER>
__device__ __forceinline__ constexpr int first_of(int e) { return INTER ? 2 * e : e; }
template <int N, bool INTER>
__device__ __forceinline__ constexpr int second_of(int e) { return INTER ? 2 * e + 1 : N + e; }

// Turned by the angles, or back by them (BACK).
template <int N, bool INTER, bool BACK>
__device__ __forceinline__ void turn(const float2 *angles, float (&v)[2 * N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float2 t = angles[e];
    const float s = BACK ? -t.y : t.y;
    float &a = v[first_of<N, INTER>(e)], &b = v[second_of<N, INTER>(e)];
    const float x = a, y = b;
    a = __builtin_fmaf(x, t.x, -(y * s));
    b = __builtin_fmaf(x, s, y * t.x);
  }
}

// Sum over the lanes of a row (a power of two of them), in every lane.
__device__ __forceinline__ double row_sum(double v, int lanes) {
  if (lanes > 1) v += lane_xor<1>(v);
  if (lanes > 2) v += lane_xor<2>(v);
  if (lanes > 4) v += lane_xor<7>(v);
  if (lanes > 8) v += lane_xor<15>(v);
  if (lanes > 16) v += lane_xor<16>(v);
  return v;
}

// v *= 1 / rms, in float32 where that is a normal number.  Rows of 3e-39 or of 1e38 with
// an eps that is no larger have a reciprocal beyond, and so has any row of zeros with an
// eps below 1e-77, though the products are numbers: those are made in 64 bits.
template <int N>
__device__ __forceinline__ void times_inverse(float (&v)[2 * N], double inv) {
  const float u = (float)inv;
  if (__builtin_isnormal(u)) {
#pragma unroll
    for (int e = 0; e < 2 * N; ++e) v[e] *= u;
  } else {
#pragma unroll
    for (int e = 0; e < 2 * N; ++e) {
      float x = v[e];
      asm volatile("" : "+v"(x));   // (else the sum's 64-bit elements are kept for here)
      v[e] = (float)((double)x * inv);
    }
  }
}

__device__ __forceinline__ void make_turns(const RopeParams &p, int64_t token0, int tokens,
                                           float2 *turns) {
  for (int i = threadIdx.x; i < tokens * p.pairs; i += kThreads) {
    const int t = i / p.pairs, j = i - t * p.pairs;
    turns[i] = turn_of(p.positions[token0 + t], p.freqs[j]);
  }
}

template <typename T, int N, bool INTER>
__device__ __forceinline__ void forward_rows(const RopeParams &p, const RopeSide &side,
                                             int64_t token0, int tokens, int lanes,
                                             const Slot<N> &s, const float2 *turns) {
  using S = typename T::S;
  if (side.heads == 0) return;
  float w[2 * N];
#pragma unroll
  for (int e = 0; e < 2 * N; ++e)
    w[e] = s.there && side.weight ? side.weight[e < N ? s.lo + e : s.hi + e - N] : 1.0f;
  const int rows = tokens * side.heads, step = kThreads / lanes;
  for (int r = threadIdx.x / lanes; r - (int)threadIdx.x / lanes < rows; r += step) {
    const bool on = s.there && r < rows;
    const int t = r / side.heads, h = r - t * side.heads;
    float v[2 * N];
#pragma unroll
    for (int e = 0; e < 2 * N; ++e) v[e] = 0.0f;
    if (on)
      load_slot<T, N>((const S *)side.x + (token0 + t) * side.x_token + h * side.x_head, s, v);
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < 2 * N; ++e) sum = __builtin_fma((double)v[e], (double)v[e], sum);
    const double inv = 1.0 / sqrt(row_sum(sum, lanes) / p.dim + p.eps);
    if (on) {
      times_inverse<N>(v, inv);
#pragma unroll
      for (int e = 0; e < 2 * N; ++e) v[e] *= w[e];
      if (s.turned) turn<N, INTER, false>(turns + t * p.pairs + s.pair, v);
      store_slot<T, N>((S *)side.y + (token0 + t) * side.y_token + h * side.y_head, s, v);
    }
  }
}

template <typename T, int N, bool INTER, int TOKENS>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p, int lanes, int each) {
  __shared__ float2 turns[TOKENS * kMaxPairs];
  const Slot<N> s = slot_of<N, INTER>(threadIdx.x & (lanes - 1), p.dim, p.pairs);
  for (int64_t t0 = (int64_t)blockIdx.x * each; t0 < p.tokens;
       t0 += (int64_t)gridDim.x * each) {
    const int tokens = (int)(p.tokens - t0 < each ? p.tokens - t0 : each);
    make_turns(p, t0, tokens, turns);
    __syncthreads();
    forward_rows<T, N, INTER>(p, p.q, t0, tokens, lanes, s, turns);
    forward_rows<T, N, INTER>(p, p.k, t0, tokens, lanes, s, turns);
    __syncthreads();
  }
}

template <typename T, int N, bool INTER>
__device__ __forceinline__ void backward_rows(const RopeParams &p, const RopeSide &side,
                                              int64_t token0, int tokens, int lanes,
                                              const Slot<N> &s, const float2 *turns,
                                              const float (&w)[2 * N], float (&dw)[2 * N]) {
  using S = typename T::S;
  if (side.heads == 0) return;
  const int rows = tokens * side.heads, step = kThreads / lanes;
  for (int r = threadIdx.x / lanes; r - (int)threadIdx.x / lanes < rows; r += step) {
    const bool on = s.there && r < rows;
    const int t = r / side.heads, h = r - t * side.heads;
    float v[2 * N], d[2 * N];
#pragma unroll
    for (int e = 0; e < 2 * N; ++e) v[e] = d[e] = 0.0f;
    if (on) {
      load_slot<T, N>((const S *)side.x + (token0 + t) * side.x_token + h * side.x_head, s, v);
      load_slot<T, N>((const S *)side.grad + (token0 + t) * side.g_token + h * side.g_head, s, d);
      if (s.turned) turn<N, INTER, true>(turns + t * p.pairs + s.pair, d);
    }
    double sum = 0.0, dot = 0.0;
#pragma unroll
    for (int e = 0; e < 2 * N; ++e) {
      sum = __builtin_fma((double)v[e], (double)v[e], sum);
      dot = __builtin_fma((double)(d[e] * w[e]), (double)v[e], dot);
    }
    const double inv = 1.0 / sqrt(row_sum(sum, lanes) / p.dim + p.eps);
    const float along = (float)(row_sum(dot, lanes) * inv / p.dim);   // mean(g u)
    if (on) {
      times_inverse<N>(v, inv);
#pragma unroll
      for (int e = 0; e < 2 * N; ++e) {
        dw[e] = __builtin_fmaf(d[e], v[e], dw[e]);
        v[e] = __builtin_fmaf(-v[e], along, d[e] * w[e]);
      }
      times_inverse<N>(v, inv);
      store_slot<T, N>((S *)side.y + (token0 + t) * side.y_token + h * side.y_head, s, v);
    }
  }
}

// A workgroup's share of the weights' gradients: its rows' sums, added over the
// groups of lanes in a fixed order.
template <int N>
__device__ __forceinline__ void put_weight_sums(const float (&dw)[2 * N], const Slot<N> &s,
                                                int dim, int lanes, float *sums, float *to) {
  const int groups = kThreads / lanes, group = threadIdx.x / lanes;
  __syncthreads();
  for (int g0 = 0; g0 < groups; g0 += 8) {   // eight rows of `sums` at a time
    if (s.there && group >= g0 && group < g0 + 8) {
#pragma unroll
      for (int e = 0; e < 2 * N; ++e) {
        float *at = sums + (group - g0) * kMaxRopeDim + (e < N ? s.lo + e : s.hi + e - N);
        *at = g0 ? *at + dw[e] : dw[e];
      }
    }
    __syncthreads();
  }
  const int have = groups < 8 ? groups : 8;
  for (int i = threadIdx.x; i < dim; i += kThreads) {
    float a = 0.0f;
    for (int g = 0; g < have; ++g) a += sums[g * kMaxRopeDim + i];
    to[i] = a;
  }
  __syncthreads();
}

template <typename T, int N, bool INTER, int TOKENS>
__global__ __launch_bounds__(kThreads) void rope_grad_kernel(RopeParams p, int lanes,
                                                             int each, float *partial) {
  __shared__ float2 turns[TOKENS * kMaxPairs];
  __shared__ float sums[8 * kMaxRopeDim];
  const Slot<N> s = slot_of<N, INTER>(threadIdx.x & (lanes - 1), p.dim, p.pairs);
  float wq[2 * N], wk[2 * N], dq[2 * N], dk[2 * N];
#pragma unroll
  for (int e = 0; e < 2 * N; ++e) {
    const int at = e < N ? s.lo + e : s.hi + e - N;
    wq[e] = s.there && p.q.weight ? p.q.weight[at] : 1.0f;
    wk[e] = s.there && p.k.weight ? p.k.weight[at] : 1.0f;
    dq[e] = dk[e] = 0.0f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * each; t0 < p.tokens;
       t0 += (int64_t)gridDim.x * each) {
    const int tokens = (int)(p.tokens - t0 < each ? p.tokens - t0 : each);
    make_turns(p, t0, tokens, turns);
    __syncthreads();
    backward_rows<T, N, INTER>(p, p.q, t0, tokens, lanes, s, turns, wq, dq);
    backward_rows<T, N, INTER>(p, p.k, t0, tokens, lanes, s, turns, wk, dk);
    __syncthreads();
  }
  float *to = partial + (int64_t)blockIdx.x * 2 * p.dim;
  if (p.q.dweight) put_weight_sums<N>(dq, s, p.dim, lanes, sums, to);
  if (p.k.dweight) put_weight_sums<N>(dk, s, p.dim, lanes, sums, to + p.dim);
}

// dweight[i] = the sum of the workgroups' shares, in 64 bits and a fixed order:
// 16 elements a workgroup, its threads 64 shares at a time.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void rope_weight_kernel(const float *partial, int blocks,
                                                                  int dim, float *dq, float *dk) {
  constexpr int GROUPS = kSumThreads / 16;
  __shared__ double part[GROUPS][16];
  float *out = blockIdx.y ? dk : dq;
  if (!out) return;
  const int e = threadIdx.x & 15, i = blockIdx.x * 16 + e, g = threadIdx.x / 16;
  double a = 0.0;
  if (i < dim) {
#pragma unroll 4
    for (int b = g; b < blocks; b += GROUPS)
      a += (double)partial[((int64_t)b * 2 + blockIdx.y) * dim + i];
  }
  part[g][e] = a;
  __syncthreads();
  for (int half = GROUPS / 2; half > 0; half /= 2) {
    if (g < half) part[g][e] += part[g + half][e];
    __syncthreads();
  }
  if (g == 0 && i < dim) out[i] = (float)part[0][e];
}

constexpr int kGradBlocks = 512;   // two a CU
constexpr int kBlockTokens = 4;

// Several tokens a workgroup share the heads evenly over its lanes; few tokens
// take a workgroup each.
bool many(int64_t tokens) { return tokens >= 1024; }

// Four tokens or more, where few and short rows would leave lanes without one (28785
// tokens of 4 + 2 heads of 8 in bfloat16: 12 us for 18, gradient 24 for 51; 100000 of
// 1 + 1 of 64 34 for 105 and 63 for 182): as many as LDS holds the turns of, and
// workgroups are left for all CUs.  (The last of these still use 64 of the 256 threads,
// 16 tokens of 4 lanes, for q and again for k.)
int tokens_each(const RopeParams &p, int lanes) {
  if (!many(p.tokens)) return 1;
  const int heads = p.q.heads > p.k.heads ? p.q.heads : p.k.heads;
  int each = kBlockTokens;
  while ((int64_t)each * heads * lanes < kThreads && each * 2 * p.pairs <= kBlockTokens * kMaxPairs &&
         p.tokens / (each * 2) >= kGradBlocks)
    each *= 2;
  return each;
}
int grad_blocks(int64_t tokens, int each) {
  const int64_t b = (tokens + each - 1) / each;
  return (int)(b < kGradBlocks ? b : kGradBlocks);
}

template <typename F>
void each_kind(const RopeParams &p, F &&f) {
  // eight elements at a time where the pairs and the row allow it: 16 bytes of
  // bfloat16 a load
  const bool wide = p.pairs % 8 == 0 && p.dim % 16 == 0;
  int lanes = 1;
  while (lanes < p.dim / (wide ? 16 : 8)) lanes *= 2;
  f(wide, lanes);
}

template <typename T, int N, bool INTER>
hipError_t run_forward(const RopeParams &p, int lanes, hipStream_t stream) {
  const int each = tokens_each(p, lanes);
  const int64_t blocks = (p.tokens + each - 1) / each;
  const uint32_t grid = (uint32_t)(blocks < (1 << 22) ? blocks : 1 << 22);
  if (many(p.tokens))
    launch_kernel(rope_kernel<T, N, INTER, kBlockTokens>, dim3(grid), dim3(kThreads), 0, stream, p,
                  lanes, each);
  else
    launch_kernel(rope_kernel<T, N, INTER, 1>, dim3(grid), dim3(kThreads), 0, stream, p, lanes, each);
  return hipGetLastError();
}

template <typename T, int N, bool INTER>
hipError_t run_backward(const RopeParams &p, int lanes, float *partial, hipStream_t stream) {
  const int each = tokens_each(p, lanes), blocks = grad_blocks(p.tokens, each);
  if (many(p.tokens))
    launch_kernel(rope_grad_kernel<T, N, INTER, kBlockTokens>, dim3(blocks), dim3(kThreads), 0,
                  stream, p, lanes, each, partial);
  else if (p.tokens)
    launch_kernel(rope_grad_kernel<T, N, INTER, 1>, dim3(blocks), dim3(kThreads), 0, stream, p,
                  lanes, each, partial);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.q.dweight && !p.k.dweight)) return e;
  launch_kernel(rope_weight_kernel, dim3((p.dim + 15) / 16, 2), dim3(kSumThreads), 0,
                stream, (const float *)partial, blocks, p.dim, p.q.dweight, p.k.dweight);
  return hipGetLastError();
}

}  // namespace

size_t rope_grad_workspace(int64_t tokens, int dim) {
  return (size_t)grad_blocks(tokens, many(tokens) ? kBlockTokens : 1) * 2 * dim * sizeof(float);
}

hipError_t launch_rope(const RopeParams &p, int dtype, bool interleaved, hipStream_t stream) {
  hipError_t e = hipSuccess;
  each_kind(p, [&](bool wide, int lanes) {
#define DLRM_ROPE(T)                                                                         \
  e = wide ? (interleaved ? run_forward<T, 8, true>(p, lanes, stream)                        \
                          : run_forward<T, 8, false>(p, lanes, stream))                      \
           : (interleaved ? run_forward<T, 4, true>(p, lanes, stream)                        \
                          : run_forward<T, 4, false>(p, lanes, stream))
    if (dtype == kF32)
      DLRM_ROPE(F32);
    else
      DLRM_ROPE(BF16);
#undef DLRM_ROPE
  });
  return e;
}

hipError_t launch_rope_grad(const RopeParams &p, int dtype, bool interleaved, void *ws,
                            hipStream_t stream) {
  hipError_t e = hipSuccess;
  float *partial = (float *)ws;
  each_kind(p, [&](bool wide, int lanes) {
#define DLRM_ROPE(T)                                                                         \
  e = wide ? (interleaved ? run_backward<T, 8, true>(p, lanes, partial, stream)              \
                          : run_backward<T, 8, false>(p, lanes, partial, stream))            \
           : (interleaved ? run_backward<T, 4, true>(p, lanes, partial, stream)              \
                          : run_backward<T, 4, false>(p, lanes, partial, stream))
    if (dtype == kF32)
      DLRM_ROPE(F32);
    else
      DLRM_ROPE(BF16);
#undef DLRM_ROPE
  });
  return e;
}

}  // namespace dlrm
