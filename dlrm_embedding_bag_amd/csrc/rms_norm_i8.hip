// rms_norm_i8.hip -- residual addition, RMS norm and int8 quantisation of
// rows in one launch:
//
//   h = round(x + residual)            (the rows' type)
//   y = h * weight / sqrt(mean(h^2) + eps)
//   s = max|y| / 127                   (float32, one per row)
//   q = round(y / s)                   (int8, ties to even)
//
// Codes are whole numbers that a consumer multiplies exactly, so each is
// decided in 64 bits: the sum of squares, the products h * weight (exact: 24
// by 24 bits), the maximum and y / s are float64.  A float64 multiply-add has
// float32's rate on this chip, and the kernel stays bound by memory.
//
// A row is held in registers between its two uses (statistics, codes), so
// memory is read and written once: 2 reads and 1 write of the rows' type,
// one byte of code per element.
#include <math.h>

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

// Sum and maximum over the TPR threads of a row (whole waves); every thread
// ends with both.  `sh` holds two doubles per wave of the workgroup.
template <int TPR>
__device__ __forceinline__ void row_reduce(double &ss, double &mx, double *sh, int lane_in_row) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    ss += __shfl_xor(ss, o);
    mx = fmax(mx, __shfl_xor(mx, o));
  }
  if constexpr (TPR > kWave) {
    constexpr int W = TPR / kWave;
    const int w = lane_in_row / kWave;
    if (lane_in_row % kWave == 0) {
      sh[2 * w] = ss;
      sh[2 * w + 1] = mx;
    }
    __syncthreads();
    ss = sh[0];
    mx = sh[1];
#pragma unroll
    for (int i = 1; i < W; ++i) {
      ss += sh[2 * i];
      mx = fmax(mx, sh[2 * i + 1]);
    }
  }
}

// What a row's statistics give its codes: the float32 scale, and the factor
// of h * weight in float64 (zero when the row has no codes: all zero, or a
// scale that is not finite).
struct RowScale {
  float s;
  double f;
};
__device__ __forceinline__ RowScale row_scale(double ss, double mx, int dim, double eps) {
  // an infinite sum (an infinity in the row) leaves no value, also where every
  // product h * weight that is compared is finite
  const double r = ss < INFINITY ? 1.0 / sqrt(ss / dim + eps) : NAN;
  RowScale o;
  o.s = (float)(mx * r / 127.0);
  o.f = (o.s > 0.0f && o.s < INFINITY) ? r / (double)o.s : 0.0;
  return o;
}

__device__ __forceinline__ int code(float h, float w, double f) {
  const double v = rint((double)h * (double)w * f);
  return (int)fmin(fmax(v, -127.0), 127.0);
}

__device__ __forceinline__ void store_codes(int8_t *row, int c, int dim, const float (&h)[8],
                                            const float (&w)[8], double f) {
  int q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = f != 0.0 ? code(h[e], w[e], f) : 0;
  if (c + 8 <= dim) {
    u32x2_u v;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      v[e] = (q[4 * e] & 255) | (q[4 * e + 1] & 255) << 8 | (q[4 * e + 2] & 255) << 16 |
             (uint32_t)q[4 * e + 3] << 24;
    *reinterpret_cast<u32x2_u *>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < dim) row[c + e] = (int8_t)q[e];
  }
}

// One chunk of h: x (+ residual, rounded to the rows' type).
template <typename T, bool RES>
__device__ __forceinline__ void load_h(const NormParams &p, int64_t m, int c, float (&h)[8]) {
  using S = typename T::S;
  load_chunk<T>((const S *)p.x + m * p.ldx, c, p.dim, h);
  if (RES) {
    float r[8];
    load_chunk<T>((const S *)p.residual + m * p.ldr, c, p.dim, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[e] += r[e];
      if constexpr (sizeof(S) == 2) h[e] = __uint_as_float((uint32_t)to_bf16(h[e]) << 16);
    }
  }
}

__device__ __forceinline__ void load_w(const float *w, int c, int dim, float (&v)[8]) {
  if (w) {
    load_chunk<F32>(w, c, dim, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
  }
}

__device__ __forceinline__ void accumulate(const float (&h)[8], const float (&w)[8], double &ss,
                                           double &mx, float &bad) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double d = h[e];
    ss = __builtin_fma(d, d, ss);
    mx = fmax(mx, fabs(d * (double)w[e]));
    bad = __builtin_fmaf(w[e], 0.0f, bad);
  }
}

// TPR threads hold a row of up to TPR * 8 * NV elements.
template <typename T, bool RES, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormParams p) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ double sh[2 * (TPR / kWave)];
  const int t = threadIdx.x % TPR;
  for (int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; m < p.m;
       m += (int64_t)gridDim.x * RPB) {
    float h[NV][8], w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c < p.dim) load_h<T, RES>(p, m, c, h[i]);
    }
    double ss = 0.0, mx = 0.0;
    float bad = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c < p.dim) {
        load_w(p.weight, c, p.dim, w[i]);
        if (RES) store_chunk<T>((typename T::S *)p.h + m * p.ldh, c, p.dim, h[i]);
        accumulate(h[i], w[i], ss, mx, bad);
      }
    }
    // a weight that is not finite makes the row's sum NaN, and so its scale
    ss += bad;
    row_reduce<TPR>(ss, mx, sh, t);
    const RowScale rs = row_scale(ss, mx, p.dim, p.eps);
    if (t == 0) p.scale[m] = rs.s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c < p.dim) store_codes(p.codes + m * p.ldq, c, p.dim, h[i], w[i], rs.f);
    }
    if (TPR > kWave) __syncthreads();  // sh is read before the next row writes it
  }
}

// Rows longer than any register form: each thread reads its chunks again for
// the codes (h from where it stored them itself).
template <typename T, bool RES>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormParams p) {
  __shared__ double sh[2 * (1024 / kWave)];
  for (int64_t m = blockIdx.x; m < p.m; m += gridDim.x) {
    double ss = 0.0, mx = 0.0;
    float bad = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.dim; c += 1024 * 8) {
      float h[8], w[8];
      load_h<T, RES>(p, m, (int)c, h);
      load_w(p.weight, (int)c, p.dim, w);
      if (RES) store_chunk<T>((typename T::S *)p.h + m * p.ldh, (int)c, p.dim, h);
      accumulate(h, w, ss, mx, bad);
    }
    ss += bad;
    row_reduce<1024>(ss, mx, sh, threadIdx.x);
    const RowScale rs = row_scale(ss, mx, p.dim, p.eps);
    if (threadIdx.x == 0) p.scale[m] = rs.s;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < p.dim; c += 1024 * 8) {
      float h[8], w[8];
      if (RES)
        load_chunk<T>((const typename T::S *)p.h + m * p.ldh, (int)c, p.dim, h);
      else
        load_chunk<T>((const typename T::S *)p.x + m * p.ldx, (int)c, p.dim, h);
      load_w(p.weight, (int)c, p.dim, w);
      store_codes(p.codes + m * p.ldq, (int)c, p.dim, h, w, rs.f);
    }
    __syncthreads();
  }
}

template <typename T, bool RES>
hipError_t launch_typed(const NormParams &p, hipStream_t stream) {
  // a launch holds fewer than 2^32 threads; the workgroups loop over the rest
  const unsigned m = (unsigned)(p.m < (1 << 21) ? p.m : 1 << 21);
  if (p.dim <= 512)
    launch_kernel(norm_kernel<T, RES, 64, 1>, dim3((m + 3) / 4), dim3(256), 0, stream, p);
  else if (p.dim <= 2048)
    launch_kernel(norm_kernel<T, RES, 256, 1>, dim3(m), dim3(256), 0, stream, p);
  else if (p.dim <= 4096)
    launch_kernel(norm_kernel<T, RES, 256, 2>, dim3(m), dim3(256), 0, stream, p);
  else if (p.dim <= 8192)
    launch_kernel(norm_kernel<T, RES, 256, 4>, dim3(m), dim3(256), 0, stream, p);
  else
    launch_kernel(norm_long_kernel<T, RES>, dim3(m), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm_i8(const NormParams &p, int dtype, hipStream_t stream) {
  if (dtype == kBF16)
    return p.residual ? launch_typed<BF16, true>(p, stream) : launch_typed<BF16, false>(p, stream);
  return p.residual ? launch_typed<F32, true>(p, stream) : launch_typed<F32, false>(p, stream);
}

}  // namespace dlrm
