// kv_cache.hip -- keys and values quantised as they are written into a paged
// cache, and read back.
//
// A row's 32 values share a power of two, kept as its exponent plus 127: the
// smallest 2^e that clips none of them,
//   e = the least e >= -117 with max |x| <= 448 * 2^e  (8 bits: E4M3 codes)
//                               or  <= 6 * 2^e         (4 bits: E2M1 codes)
// (but at most 119 or 125, where magnitudes beyond 1.75 or 1.5 * 2^127 are clipped
// to them: no value that codes stand for is an infinity in float32 or bfloat16),
// so that x 2^-e rounds to the nearest code, ties to the even one, by the
// conversion instructions, which take the scale along.  With e >= -117 every
// value that codes stand for is zero or a normal number of bfloat16, too.  A
// group that holds an infinity or a NaN has the scale 255, which reads as NaN.
//
// A lane takes eight values; four lanes share a group.  Bounded by memory: rows
// are read or written in pieces of 16 bytes or more a lane, codes in 8 or 4.
// (16384 tokens of 8 heads of 128 in bfloat16 and 8 bits: written in 27 us, 3.7 TB/s,
// read in 19, 5.3 TB/s, out of the caches in part.)
#include "cache_common.hpp"

namespace dlrm {
namespace {

constexpr int kThreads = 256;
typedef short i16x2_t __attribute__((ext_vector_type(2)));

// Where eight values of a row go, or come from.
struct Place {
  int64_t token, row;  // row: of the cache; -1 where there is none
  int head, chunk;     // of eight values
};

__device__ __forceinline__ Place place_of(const CacheParams &p, int64_t i, int chunk_bits) {
  Place at;
  at.chunk = (int)i & ((1 << chunk_bits) - 1);
  const int64_t th = i >> chunk_bits;
  at.token = th / p.heads;
  at.head = (int)(th - at.token * p.heads);
  const int32_t slot = p.slots[at.token];
  const int page_bits = 31 - __clz(p.page);
  const bool there = slot >= 0 && (slot >> page_bits) < p.pages;
  at.row = there ? ((int64_t)(slot >> page_bits) * p.heads + at.head) * p.page +
                       (slot & (p.page - 1))
                 : -1;
  return at;
}

template <typename T, int BITS>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheParams p, int chunk_bits,
                                                               int64_t items) {
  using S = typename T::S;
  const bool values = blockIdx.y;
  const S *x = (const S *)(values ? p.v : p.k);
  const int64_t xt = values ? p.v_token : p.k_token, xh = values ? p.v_head : p.k_head;
  uint8_t *codes = values ? p.v_codes : p.k_codes, *scales = values ? p.v_scales : p.k_scales;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads; i0 < items;
       i0 += (int64_t)gridDim.x * kThreads) {
    const int64_t i = i0 + threadIdx.x;
    const bool on = i < items;   // a row's lanes are on or off together
    const Place at = place_of(p, on ? i : items - 1, chunk_bits);
    float v[8];
    load8<T>(x + at.token * xt + at.head * xh + at.chunk * 8, v);
    uint32_t top = 0;            // of the magnitudes' bits; infinities and NaN above all
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t a = __float_as_uint(v[e]) & 0x7fffffffu;
      top = top > a ? top : a;
    }
    uint32_t o = lane_xor<1>(top);
    top = top > o ? top : o;
    o = lane_xor<2>(top);
    top = top > o ? top : o;
    if (!on || at.row < 0) continue;
    // 448 = 1.75 * 2^8, 6 = 1.5 * 2^2
    const uint32_t most = BITS == 8 ? 0x600000u : 0x400000u;
    int scale = (int)(top >> 23) - (BITS == 8 ? 8 : 2) + ((top & 0x7fffffu) > most);
    constexpr int kMax = BITS == 8 ? 119 + 127 : 125 + 127;
    scale = scale < kMinScale ? kMinScale : scale > kMax ? kMax : scale;
    const float clip = __uint_as_float(0x7f000000u | most);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(v[e], -clip), clip);
    const bool bad = top >= 0x7f800000u;
    const float unit = __uint_as_float((uint32_t)scale << 23);
    uint8_t *to = codes + at.row * (p.dim * BITS / 8) + at.chunk * BITS;
    if constexpr (BITS == 8) {
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        i16x2_t r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * e], v[4 * e + 1], unit, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * e + 2], v[4 * e + 3], unit, true);
        w[e] = bad ? 0u : __builtin_bit_cast(uint32_t, r);
      }
      *reinterpret_cast<u32x2_u *>(to) = u32x2_u{w[0], w[1]};
    } else {
      uint32_t w = 0;
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], unit, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], unit, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], unit, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], unit, 3);
      *reinterpret_cast<u32_u *>(to) = bad ? 0u : w;
    }
    if ((at.chunk & 3) == 0)
      scales[at.row * (p.dim / kGroup) + at.chunk / 4] = bad ? 255 : (uint8_t)scale;
  }
}

template <typename T, int BITS>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheParams p, int chunk_bits,
                                                              int64_t items) {
  using S = typename T::S;
  const bool values = blockIdx.y;
  S *x = (S *)(values ? p.out_v : p.out_k);
  const int64_t xt = values ? p.v_token : p.k_token, xh = values ? p.v_head : p.k_head;
  const uint8_t *codes = values ? p.v_codes : p.k_codes;
  const uint8_t *scales = values ? p.v_scales : p.k_scales;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * kThreads) {
    const Place at = place_of(p, i, chunk_bits);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (at.row >= 0) {
      const float unit =
          unit_of(scales[at.row * (p.dim / kGroup) + at.chunk / 4]);
      const uint8_t *from = codes + at.row * (p.dim * BITS / 8) + at.chunk * BITS;
      Codes<BITS> c;
      if constexpr (BITS == 8) {
        const u32x2_u w = *reinterpret_cast<const u32x2_u *>(from);
        c.w[0] = w[0];
        c.w[1] = w[1];
      } else {
        c.w[0] = *reinterpret_cast<const u32_u *>(from);
      }
      values_of(c, unit, v);
    }
    store8<T>(x + at.token * xt + at.head * xh + at.chunk * 8, v);
  }
}

template <bool WRITE, typename T, int BITS>
hipError_t run(const CacheParams &p, hipStream_t stream) {
  int chunk_bits = 0;
  while ((8 << chunk_bits) < p.dim) ++chunk_bits;
  const int64_t items = (p.tokens * p.heads) << chunk_bits;
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)(blocks < (1 << 22) ? blocks : 1 << 22), 2);
  if constexpr (WRITE)
    launch_kernel(cache_write_kernel<T, BITS>, grid, dim3(kThreads), 0, stream, p, chunk_bits,
                  items);
  else
    launch_kernel(cache_read_kernel<T, BITS>, grid, dim3(kThreads), 0, stream, p, chunk_bits,
                  items);
  return hipGetLastError();
}

template <bool WRITE>
hipError_t by_type(const CacheParams &p, int dtype, int bits, hipStream_t stream) {
  if (dtype == kF32)
    return bits == 8 ? run<WRITE, F32, 8>(p, stream) : run<WRITE, F32, 4>(p, stream);
  return bits == 8 ? run<WRITE, BF16, 8>(p, stream) : run<WRITE, BF16, 4>(p, stream);
}

}  // namespace

hipError_t launch_cache_write(const CacheParams &p, int dtype, int bits, hipStream_t stream) {
  return by_type<true>(p, dtype, bits, stream);
}
hipError_t launch_cache_read(const CacheParams &p, int dtype, int bits, hipStream_t stream) {
  return by_type<false>(p, dtype, bits, stream);
}

}  // namespace dlrm
