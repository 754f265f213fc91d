// rms_norm_i8.hip -- residual addition, RMS norm and int8 quantisation of
// rows in one launch:
//
//   h = round(x + residual)            (the rows' type)
//   y = h * weight / sqrt(mean(h^2) + eps)
//   s = max|y| / 127                   (float32, one per row)
//   q = round(y / s)                   (int8, ties to even)
//
// Codes are whole numbers that a consumer multiplies exactly, so each is the
// one that 64 bits decide: the sum of squares, the products h * weight (exact:
// 24 by 24 bits) and their maximum are float64, whose instructions have
// float32's rate on this chip; y / s in float32 decides a code unless it lies
// within 2^-14 of a border, where float64 does.
//
// A row is held in registers between its two uses (statistics, codes), so
// memory is read and written once: 2 reads and 1 write of the rows' type, one
// byte of code per element, written past the caches (4096 rows' h and codes
// otherwise push out inputs: 110 us for 79).  Memory bounds rows of up to 4096:
// 16384 rows of 4096 float32 with a residual take 157 us, 5.6 TB/s, 32768 of
// bfloat16 176 us, 5.3 TB/s.  16384 bfloat16 rows of 8192, the same bytes, take
// 201 us, 4.7 TB/s: their waits for a row's sum between loads and stores are not
// all covered by the three rows that a CU holds (its waves wait 73% of their
// time).  Longer rows are read again for the codes: 8192 rows of 12288 take 243
// us, 2.9 TB/s, of 16384 289 us, 3.3 TB/s.
#include <math.h>

#include <type_traits>

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

// Lanes of a wave that share a row with TPR threads.
template <int TPR>
constexpr int lanes_of_row() {
  return TPR < kWave ? TPR : kWave;
}

// Sum and maximum over 2 X lanes.
template <int X>
__device__ __forceinline__ void lanes_reduce(double &ss, double &mx) {
  if constexpr (X > 0) {
    lanes_reduce<X / 2>(ss, mx);
    ss += lane_xor<X>(ss);
    mx = fmax(mx, lane_xor<X>(mx));
  }
}

// Sum and maximum over the TPR threads of a row (a part of a wave, or whole
// waves); every thread ends with both.  `sh` holds two doubles per wave.
template <int TPR>
__device__ __forceinline__ void row_reduce(double &ss, double &mx, double *sh, int lane_in_row) {
  lanes_reduce<lanes_of_row<TPR>() / 2>(ss, mx);
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

// Products h * weight between this and its inverse are rounded to float32, and
// scaled, without leaving its normal range (beyond it a product overflows).
constexpr double kLeast = 0x1p-100;
// float32's least normal value: a scale below it has fewer than 24 bits, and
// max|y| / scale may lie well beyond 127.
constexpr float kLeastScale = 0x1p-126f;

// 1 / sqrt(d) and 1 / d in float64: the hardware's estimate and two steps of
// Newton's iteration, each of which doubles its digits (24 at least).  Every
// thread of a row computes them, and the library's exact ones took longer than
// a short row's codes.
__device__ __forceinline__ double inverse_root(double d) {
  double y = __builtin_amdgcn_rsq(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(0.5 * y, __builtin_fma(-d * y, y, 1.0), y);
  return y;
}
__device__ __forceinline__ double inverse(double d) {
  double y = __builtin_amdgcn_rcp(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
  return y;
}

// What a row's statistics give its codes: the float32 scale, and the factor
// of h * weight in float64 (zero when the row has no codes: all zero, or a
// scale that is not finite).
struct RowScale {
  float s;
  double f;
  float f32;  // f where float32 decides most codes, else 0
};
__device__ __forceinline__ RowScale row_scale(double ss, double mx, int dim, double eps) {
  // an infinite sum (an infinity in the row) leaves no value, also where every
  // product h * weight that is compared is finite
  const double r = ss < INFINITY ? inverse_root(ss / dim + eps) : NAN;
  RowScale o;
  o.s = (float)(mx * r * (1.0 / 127.0));
  o.f = (o.s > 0.0f && o.s < INFINITY) ? r * inverse((double)o.s) : 0.0;
  o.f32 = mx > kLeast && mx < 1.0 / kLeast && o.s >= kLeastScale ? (float)o.f : 0.0f;
  return o;
}

__device__ __forceinline__ int code(float h, float w, double f) {
  const double v = rint((double)h * (double)w * f);
  return (int)fmin(fmax(v, -127.0), 127.0);
}

__device__ __forceinline__ void store_codes(int8_t *row, int c, int dim, const float (&h)[8],
                                            const float (&w)[8], const RowScale &rs) {
  // Added to 1.5 * 2^23 a value is rounded to a whole number (ties to even),
  // whose low byte is the code.  Values are at most 127 but for the scale's
  // rounding, 127 * 2^-24 (f32 is zero where a scale has fewer bits).  h * w and
  // f32 are each off by at most 2^-24 of that: where a value lies 2^-14 or more
  // from a border, the exact one lies on the same side, and both round to the
  // same code.
  constexpr float kWhole = 12582912.0f;
  uint32_t q[8];
  bool clear = rs.f32 != 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float p = h[e] * w[e], t = __builtin_fmaf(p, rs.f32, kWhole);
    clear &= fabsf(__builtin_fmaf(p, rs.f32, kWhole - t)) < 0.5f - 0x1p-14f;  // (not for NaN)
    q[e] = __float_as_uint(t);
  }
  if (!clear) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = rs.f != 0.0 ? (uint32_t)code(h[e], w[e], rs.f) : 0;
  }
  if (c + 8 <= dim) {
    u32x2_u v;
#pragma unroll
    for (int e = 0; e < 2; ++e)  // the low bytes of four
      v[e] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[4 * e + 3], q[4 * e + 2], 0x0c0c0400u),
                                   __builtin_amdgcn_perm(q[4 * e + 1], q[4 * e], 0x0c0c0400u),
                                   0x05040100u);
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2_u *>(row + c));
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

// Sum of squares, largest |h * weight|; bad becomes NaN where a weight is not
// finite.
__device__ __forceinline__ void accumulate(const float (&h)[8], const float (&w)[8], double &ss,
                                           double &mx, float &bad) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double d = h[e], v = d * (double)w[e];
    ss = __builtin_fma(d, d, ss);
    // (fmax would first make both operands quiet, an instruction each)
    asm("v_max_f64 %0, %0, |%1|" : "+v"(mx) : "v"(v));
    bad = __builtin_fmaf(w[e], 0.0f, bad);
  }
}

// Rows of a workgroup: waves' rows wait for nobody, so four waves make one.
template <int TPR>
constexpr int rows_of_block() {
  return TPR <= kWave ? 256 / TPR : 1;
}

// TPR threads hold a row of up to TPR * 8 * NV elements.
template <typename T, bool RES, int TPR, int NV>
__global__ __launch_bounds__(TPR *rows_of_block<TPR>()) void norm_kernel(NormParams p) {
  constexpr int RPB = rows_of_block<TPR>();
  __shared__ double sh[TPR > kWave ? 2 * (TPR / kWave) : 1];
  const int t = threadIdx.x % TPR;
  for (int64_t m0 = (int64_t)blockIdx.x * RPB; m0 < p.m; m0 += (int64_t)gridDim.x * RPB) {
    // (lanes past the last row read it again and store nothing: lanes exchange
    // values, so all go along)
    const bool there = m0 + threadIdx.x / TPR < p.m;
    const int64_t m = there ? m0 + threadIdx.x / TPR : p.m - 1;
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
        if (RES && there)
          store_chunk<T, sizeof(typename T::S) == 2>((typename T::S *)p.h + m * p.ldh, c, p.dim,
                                                     h[i]);
        accumulate(h[i], w[i], ss, mx, bad);
      }
    }
    // a weight that is not finite makes the row's sum NaN, and so its scale
    ss += bad;
    row_reduce<TPR>(ss, mx, sh, t);
    const RowScale rs = row_scale(ss, mx, p.dim, p.eps);
    if (t == 0 && there) p.scale[m] = rs.s;
    // Where 512 threads hold a row, a CU holds few rows: the weight is read again,
    // from the caches, rather than kept, so that one row more fits (16384 rows of
    // 8192: 215 us for 235).  Shorter rows fit often enough (4096: 72 us kept,
    // 76 read again).
    constexpr bool AGAIN = TPR * NV > 512;
    const float *again = p.weight;
    if (AGAIN) asm volatile("" : "+s"(again));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * 8;
      if (c < p.dim) {
        if (AGAIN) load_w(again, c, p.dim, w[i]);
        if (there) store_codes(p.codes + m * p.ldq, c, p.dim, h[i], w[i], rs);
      }
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
      store_codes(p.codes + m * p.ldq, (int)c, p.dim, h, w, rs);
    }
    __syncthreads();
  }
}

template <int V>
using Int = std::integral_constant<int, V>;

template <typename T, bool RES>
hipError_t launch_typed(const NormParams &p, hipStream_t stream) {
  // Rows that share a wave, or a wave a row, exchange by register moves and wait
  // for nobody (65536 rows of 1024: 72 us by a wave each, 161 by 256 threads;
  // 500000 rows of 100: 88 us by 16 lanes each, 439 by a wave); a workgroup a
  // row holds a longer one in fewer registers.  Where the rows are too few to
  // fill the chip, more threads take each: one row of 4096 takes 3.4 us by 512
  // threads and 4.2 by 256.
  const bool few = p.m <= 512;
  auto launch = [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, RPB = rows_of_block<TPR>();
    // a launch holds fewer than 2^32 threads; the workgroups loop over the rest
    const int64_t blocks = (p.m + RPB - 1) / RPB, most = 1 << 21;
    launch_kernel(norm_kernel<T, RES, TPR, decltype(nv)::value>,
                  dim3((unsigned)(blocks < most ? blocks : most)), dim3(RPB * TPR), 0, stream, p);
  };
  if (p.dim <= 32)
    launch(Int<4>(), Int<1>());
  else if (p.dim <= 64)
    launch(Int<8>(), Int<1>());
  else if (p.dim <= 128)
    launch(Int<16>(), Int<1>());
  else if (p.dim <= 256)
    launch(Int<32>(), Int<1>());
  else if (p.dim <= 512)
    launch(Int<64>(), Int<1>());
  else if (p.dim <= 1024 && !few)
    launch(Int<64>(), Int<2>());
  else if (p.dim <= 2048 && !few)
    launch(Int<128>(), Int<2>());
  else if (p.dim <= 2048)
    launch(Int<256>(), Int<1>());
  else if (p.dim <= 4096)
    few ? launch(Int<512>(), Int<1>()) : launch(Int<256>(), Int<2>());
  else if (p.dim <= 8192)
    launch(Int<512>(), Int<2>());
  else
    launch_kernel(norm_long_kernel<T, RES>, dim3((unsigned)(p.m < (1 << 21) ? p.m : 1 << 21)),
                  dim3(1024), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm_i8(const NormParams &p, int dtype, hipStream_t stream) {
  if (dtype == kBF16)
    return p.residual ? launch_typed<BF16, true>(p, stream) : launch_typed<BF16, false>(p, stream);
  return p.residual ? launch_typed<F32, true>(p, stream) : launch_typed<F32, false>(p, stream);
}

}  // namespace dlrm
