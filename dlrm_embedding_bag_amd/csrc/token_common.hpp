// token_common.hpp -- internal helpers of the token operators (scaled lookup,
// its gradient, RMS norm to int8, int8 product): element types and row access.
//
// Rows of these operators may have any length and stride, so a 16-byte access
// may start at any element.  Global memory takes wide accesses at any byte
// address on this target, so one code path serves every alignment: the types
// below declare an alignment of one element (or byte) and compile to the same
// global_load_dwordx4 / global_store_dwordx4 as aligned ones.
#pragma once

#include "common.hpp"

namespace dlrm {

typedef uint32_t u32_u __attribute__((aligned(1)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(1)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Storage tags.
struct F32 { using S = float; };
struct BF16 { using S = uint16_t; };
struct FP8 { using S = uint8_t; };

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Two floats to a pair of bfloat16, each rounded once to nearest even (the
// conversion instruction of this target).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint16_t to_bf16(float a) {
  return __builtin_bit_cast(uint16_t, (__bf16)a);
}

// Eight consecutive elements as float32 (exact widening).
template <typename T>
__device__ __forceinline__ void load8(const typename T::S *p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<F32>(const float *p, float (&v)[8]) {
  const f32x4_u a = *reinterpret_cast<const f32x4_u *>(p);
  const f32x4_u b = *reinterpret_cast<const f32x4_u *>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[4 + e] = b[e];
  }
}
template <>
__device__ __forceinline__ void load8<BF16>(const uint16_t *p, float (&v)[8]) {
  const u32x4_u a = *reinterpret_cast<const u32x4_u *>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = bf16_lo(a[e]);
    v[2 * e + 1] = bf16_hi(a[e]);
  }
}
template <>
__device__ __forceinline__ void load8<FP8>(const uint8_t *p, float (&v)[8]) {
  const u32x2_u a = *reinterpret_cast<const u32x2_u *>(p);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[e], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[e], true);
    v[4 * e] = lo[0];
    v[4 * e + 1] = lo[1];
    v[4 * e + 2] = hi[0];
    v[4 * e + 3] = hi[1];
  }
}

// Four likewise.
template <typename T>
__device__ __forceinline__ void load4(const typename T::S *p, float (&v)[4]);
template <>
__device__ __forceinline__ void load4<F32>(const float *p, float (&v)[4]) {
  const f32x4_u a = *reinterpret_cast<const f32x4_u *>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = a[e];
}
template <>
__device__ __forceinline__ void load4<BF16>(const uint16_t *p, float (&v)[4]) {
  const u32x2_u a = *reinterpret_cast<const u32x2_u *>(p);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    v[2 * e] = bf16_lo(a[e]);
    v[2 * e + 1] = bf16_hi(a[e]);
  }
}
template <>
__device__ __forceinline__ void load4<FP8>(const uint8_t *p, float (&v)[4]) {
  const uint32_t a = *reinterpret_cast<const u32_u *>(p);
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)a, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)a, true);
  v[0] = lo[0];
  v[1] = lo[1];
  v[2] = hi[0];
  v[3] = hi[1];
}

template <typename T>
__device__ __forceinline__ float load1(const typename T::S *p);
template <>
__device__ __forceinline__ float load1<F32>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float load1<BF16>(const uint16_t *p) {
  return __uint_as_float((uint32_t)*p << 16);
}
template <>
__device__ __forceinline__ float load1<FP8>(const uint8_t *p) {
  return __builtin_amdgcn_cvt_f32_fp8((int)*p, 0);
}

// Eight floats to storage, each rounded once.  NT: a streaming store, for
// outputs that this kernel will not read and that would push reused rows out
// of the caches.
template <typename T, bool NT = false>
__device__ __forceinline__ void store8(typename T::S *p, const float (&v)[8]);
template <bool NT>
__device__ __forceinline__ void put16(void *p, u32x4_t v) {
  u32x4_u *q = reinterpret_cast<u32x4_u *>(p);
  if (NT)
    __builtin_nontemporal_store((u32x4_u)v, q);
  else
    *q = v;
}
template <typename T, bool NT>
__device__ __forceinline__ void store8(typename T::S *p, const float (&v)[8]) {
  if constexpr (sizeof(typename T::S) == 4) {
    u32x4_t a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = __float_as_uint(v[e]);
      b[e] = __float_as_uint(v[4 + e]);
    }
    put16<NT>(p, a);
    put16<NT>(p + 4, b);
  } else {
    u32x4_t a;
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    put16<NT>(p, a);
  }
}
template <typename T>
__device__ __forceinline__ void store1(typename T::S *p, float v) {
  if constexpr (sizeof(typename T::S) == 4)
    *p = v;
  else
    *p = to_bf16(v);
}

// Elements [c, c + N) of a row of `dim` elements (N 4 or 8); those past the row
// read as zero and are not stored.
template <typename T, int N>
__device__ __forceinline__ void load_chunk(const typename T::S *row, int c, int dim,
                                           float (&v)[N]) {
  static_assert(N == 4 || N == 8);
  if (c + N <= dim) {
    if constexpr (N == 8)
      load8<T>(row + c, v);
    else
      load4<T>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = c + e < dim ? load1<T>(row + c + e) : 0.0f;
  }
}
template <typename T, bool NT = false, int N>
__device__ __forceinline__ void store_chunk(typename T::S *row, int c, int dim,
                                            const float (&v)[N]) {
  static_assert(N == 8 || (N == 4 && sizeof(typename T::S) == 4));
  if (c + N <= dim) {
    if constexpr (N == 8) {
      store8<T, NT>(row + c, v);
    } else {
      u32x4_t a;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(v[e]);
      put16<NT>(row + c, a);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < dim) store1<T>(row + c + e, v[e]);
  }
}

// The value of lane (lane ^ X), by register moves; every lane is active.
template <int X>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  const int i = (int)v;
  if constexpr (X == 1) {          // quad_perm [1,0,3,2]
    return __builtin_amdgcn_update_dpp(0, i, 0xB1, 0xF, 0xF, true);
  } else if constexpr (X == 2) {   // quad_perm [2,3,0,1]
    return __builtin_amdgcn_update_dpp(0, i, 0x4E, 0xF, 0xF, true);
  } else if constexpr (X == 3) {   // quad_perm [3,2,1,0]
    return __builtin_amdgcn_update_dpp(0, i, 0x1B, 0xF, 0xF, true);
  } else if constexpr (X == 4) {
    return lane_xor<3>(lane_xor<7>(v));
  } else if constexpr (X == 7) {   // mirror of 8 lanes
    return __builtin_amdgcn_update_dpp(0, i, 0x141, 0xF, 0xF, true);
  } else if constexpr (X == 8) {   // rotation of 16 lanes by 8
    return __builtin_amdgcn_update_dpp(0, i, 0x128, 0xF, 0xF, true);
  } else if constexpr (X == 15) {  // mirror of 16 lanes
    return __builtin_amdgcn_update_dpp(0, i, 0x140, 0xF, 0xF, true);
  } else if constexpr (X == 16) {
    // the swap leaves the lower rows' values in one result, the upper in the other
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? r[0] : r[1];
  } else if constexpr (X == 31) {
    return lane_xor<16>(lane_xor<15>(v));
  } else if constexpr (X == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return threadIdx.x & 32 ? r[0] : r[1];
  } else {
    static_assert(X == 63);
    return lane_xor<32>(lane_xor<31>(v));
  }
}
template <int X>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
  return (uint64_t)lane_xor<X>((uint32_t)(v >> 32)) << 32 | lane_xor<X>((uint32_t)v);
}

template <int X>
__device__ __forceinline__ double lane_xor(double v) {
  return __builtin_bit_cast(double, lane_xor<X>(__builtin_bit_cast(uint64_t, v)));
}

// Eight elements as they were read, for loads that wait in registers: half the
// registers of float32 for bfloat16 rows.
template <typename T>
struct Chunk;
template <>
struct Chunk<F32> {
  float v[8];
  __device__ __forceinline__ void load(const float *row, int c, int dim) {
    load_chunk<F32>(row, c, dim, v);
  }
  __device__ __forceinline__ float at(int e) const { return v[e]; }
};
template <>
struct Chunk<BF16> {
  u32x4_t v;
  __device__ __forceinline__ void load(const uint16_t *row, int c, int dim) {
    if (c + 8 <= dim) {
      v = (u32x4_t) * reinterpret_cast<const u32x4_u *>(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = (c + 2 * e < dim ? (uint32_t)row[c + 2 * e] : 0) |
               (c + 2 * e + 1 < dim ? (uint32_t)row[c + 2 * e + 1] << 16 : 0);
    }
  }
  __device__ __forceinline__ float at(int e) const {
    return e & 1 ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
  }
};

}  // namespace dlrm
