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
#include <math.h>

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

constexpr int kBK = 128;          // bytes of k per LDS slab
constexpr int kChunks = kBK / 16;
constexpr int kXcds = 8;

__device__ __forceinline__ float apply_act(float x, int act) {
  if (act == 1) return x <= 0.0f ? 0.0f : x;  // NaN (a row without a scale) stays
  if (act == 2) return 1.0f / (1.0f + expf(-x));
  return x;
}

__device__ __forceinline__ i32x4_t load16(const int8_t *p) {
  return (i32x4_t) * reinterpret_cast<const u32x4_u *>(p);
}

// Bytes [k, k + 16) of a row of K, zeros past its end; reads stay inside the
// row (the last 16 bytes, shifted), which has at least 16 bytes or is read
// byte by byte.
__device__ __forceinline__ i32x4_t load16_tail(const int8_t *row, int k, int K) {
  if (k + 16 <= K) return load16(row + k);
  if (k >= K) return i32x4_t{0, 0, 0, 0};
  unsigned __int128 v = 0;
  if (K >= 16) {
    v = __builtin_bit_cast(unsigned __int128, load16(row + K - 16));
    v >>= 8 * (16 - (K - k));
  } else {
    for (int e = K - 1; e >= k; --e) v = v << 8 | (uint8_t)row[e];
  }
  return __builtin_bit_cast(i32x4_t, v);
}

// Four consecutive columns n.. of row m.
template <typename TO>
__device__ __forceinline__ void store_quad(const LinearI8Params &p, int m, int n, i32x4_t acc) {
  using SO = typename TO::S;
  if (m >= p.M) return;
  SO *c = (SO *)p.C + (int64_t)m * p.ldc + n;
  const float as = p.a_scale[m];
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int ne = n + e < p.N ? n + e : p.N - 1;
    v[e] = (float)acc[e] * (as * p.w_scale[ne]);
    if (p.bias) v[e] += p.bias[ne];
    v[e] = apply_act(v[e], p.act);
  }
  if (n + 4 <= p.N) {
    if constexpr (sizeof(SO) == 4) {
      *reinterpret_cast<f32x4_u *>(c) = f32x4_u{v[0], v[1], v[2], v[3]};
    } else {
      *reinterpret_cast<u32x2_u *>(c) = u32x2_u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) store1<TO>(c + e, v[e]);
  }
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
// to two LDS buffers (any alignment).  A row's 16-byte chunk c lies at place
// c ^ (row % 8) of its 128-byte row: the rows that a ds_read_b128 touches
// start on different banks.
template <int BM, int BN, int GM, int GN, typename TO>
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

  i32x4_t ra[CA], rb[CB];
  auto load = [&](int k0) {
    const bool whole = k0 + kBK <= p.K;
    const int k = k0 + cch * 16;
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int m = m0 + crow + i * (T / kChunks);
      const int8_t *row = p.A + (int64_t)(m < p.M ? m : p.M - 1) * p.lda;
      ra[i] = whole ? load16(row + k) : load16_tail(row, k, p.K);
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int n = n0 + crow + i * (T / kChunks);
      const int8_t *row = p.W + (int64_t)(n < p.N ? n : p.N - 1) * p.ldw;
      rb[i] = whole ? load16(row + k) : load16_tail(row, k, p.K);
    }
  };
  auto stage = [&](int buf) {
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

  const int slabs = (p.K + kBK - 1) / kBK;
  const int fr = lane % 16, fc = lane / 16;
  load(0);
  stage(0);
  for (int s = 0; s < slabs; ++s) {
    __syncthreads();
    if (s + 1 < slabs) load((s + 1) * kBK);
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
    if (s + 1 < slabs) stage((s + 1) & 1);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      store_quad<TO>(p, m0 + wm * (BM / GM) + i * 16 + fr, n0 + wn * (BN / GN) + j * 16 + fc * 4,
                     acc[i][j]);
}

// Few rows: bound by reading W once.  A workgroup takes 16 NF columns and all
// (up to 16 MF) rows; its 8 waves share k, 128 bytes at a time, with operands
// loaded straight into the matrix cores' layout, and add their partial tiles
// through LDS.
constexpr int kFewWaves = 8;
template <int MF, int NF, typename TO>
__global__ __launch_bounds__(kFewWaves *kWave) void few_rows_kernel(LinearI8Params p) {
  constexpr int U = 4;  // steps of 64 bytes in flight
  __shared__ i32x4_t part[kFewWaves][MF * NF][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
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
  i32x4_t acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

  const int steps = (p.K + 63) / 64;
  for (int i0 = 0;; i0 += U) {
    const int first = (i0 / 2 * kFewWaves + wave) * 2;
    if (first >= steps) break;
    i32x4_t w[U][NF], a[U][MF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int step = (u / 2 * kFewWaves) * 2 + first + u % 2;
      const int k = step * 64 + fc * 16;
      const bool whole = step * 64 + 64 <= p.K;
#pragma unroll
      for (int j = 0; j < NF; ++j)
        w[u][j] = whole ? load16(wrow[j] + k) : load16_tail(wrow[j], k, p.K);
#pragma unroll
      for (int i = 0; i < MF; ++i)
        a[u][i] = whole ? load16(arow[i] + k) : load16_tail(arow[i], k, p.K);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][j], a[u][i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) part[wave][i * NF + j][lane] = acc[i][j];
  __syncthreads();
  for (int q = threadIdx.x; q < MF * NF * kWave; q += kFewWaves * kWave) {
    const int f = q / kWave, l = q % kWave;
    i32x4_t s = part[0][f][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += part[w][f][l];
    store_quad<TO>(p, f / NF * 16 + l % 16, n0 + f % NF * 16 + l / 16 * 4, s);
  }
}

template <int BM, int BN, int GM, int GN, typename TO>
void launch_tiles(const LinearI8Params &p, hipStream_t stream) {
  const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  launch_kernel(gemm_kernel<BM, BN, GM, GN, TO>, dim3((unsigned)(tm * tn)),
                dim3(GM * GN * kWave), 0, stream, p, tm, tn);
}

template <int MF, typename TO>
void launch_few(const LinearI8Params &p, hipStream_t stream) {
  if ((p.N + 31) / 32 >= 256)
    launch_kernel(few_rows_kernel<MF, 2, TO>, dim3((p.N + 31) / 32), dim3(kFewWaves * kWave), 0,
                  stream, p);
  else
    launch_kernel(few_rows_kernel<MF, 1, TO>, dim3((p.N + 15) / 16), dim3(kFewWaves * kWave), 0,
                  stream, p);
}

template <typename TO>
hipError_t launch_typed(const LinearI8Params &p, hipStream_t stream) {
  const int64_t big = (int64_t)((p.M + 127) / 128) * ((p.N + 127) / 128);
  if (p.M <= 16)
    launch_few<1, TO>(p, stream);
  else if (p.M <= 32)
    launch_few<2, TO>(p, stream);
  else if (p.M <= 64)
    launch_few<4, TO>(p, stream);
  else if (big >= 256)
    launch_tiles<128, 128, 2, 2, TO>(p, stream);
  else
    launch_tiles<64, 64, 2, 2, TO>(p, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_i8(const LinearI8Params &p, int out_dtype, hipStream_t stream) {
  return out_dtype == kBF16 ? launch_typed<BF16>(p, stream) : launch_typed<F32>(p, stream);
}

}  // namespace dlrm
