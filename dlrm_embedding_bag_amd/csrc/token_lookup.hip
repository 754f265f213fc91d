// token_lookup.hip -- embedding lookup of single tokens with a scale:
//
//   out[t, :] = scale * table[token[t], :]     (zeros outside [0, rows))
//
// float32, bfloat16 or FP8 E4M3 rows, the product in float32, rounded once to
// the output type.  The kernel moves bytes: it is bound by the stores and by
// the distinct rows' reads.
//
// A row belongs to a group of G lanes (a power of two, up to a wave), each
// taking chunks of 8 elements; a group has kRows rows' loads in flight before
// the first store, which is what hides the token -> row chain of two memory
// round trips.  Outputs are streamed past the caches (nontemporal stores), so
// that what the caches hold is rows that other tokens will ask for.
#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

constexpr int kRows = 4;  // rows of one lane group in flight
constexpr int64_t kMaxBlocks = 1 << 22;  // a launch holds fewer than 2^32 threads

template <typename TI, typename TO>
__global__ __launch_bounds__(256) void lookup_kernel(LookupParams p, int log2g) {
  using SI = typename TI::S;
  using SO = typename TO::S;
  const int G = 1 << log2g;
  const int lane = threadIdx.x & (G - 1);
  const int64_t group = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> log2g;
  const int64_t step = (((int64_t)gridDim.x * blockDim.x) >> log2g) * kRows;
  for (int64_t t0 = group * kRows; t0 < p.tokens; t0 += step) {
    int32_t tok[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      tok[r] = t0 + r < p.tokens ? p.token[t0 + r] : -1;
    for (int c = lane * 8; c < p.dim; c += G * 8) {
      float v[kRows][8];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (tok[r] >= 0 && tok[r] < p.rows) {
          load_chunk<TI>((const SI *)p.table + (int64_t)tok[r] * p.ld_table, c, p.dim, v[r]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[r][e] = 0.0f;
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (t0 + r < p.tokens) {
          // a row that is not there is zero whatever the scale is
          const bool there = tok[r] >= 0 && tok[r] < p.rows;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[r][e] = there ? v[r][e] * p.scale : 0.0f;
          store_chunk<TO, true>((SO *)p.out + (t0 + r) * p.ld_out, c, p.dim, v[r]);
        }
      }
    }
  }
}

template <typename TI>
hipError_t launch_out(const LookupParams &p, int out_dtype, hipStream_t stream) {
  int log2g = 0;
  while ((8 << log2g) < p.dim && log2g < 6) ++log2g;
  const int64_t groups = (p.tokens + kRows - 1) / kRows;
  const int64_t want = ((groups << log2g) + 255) / 256;
  const int64_t blocks = want < kMaxBlocks ? want : kMaxBlocks;
  if (out_dtype == kBF16)
    launch_kernel(lookup_kernel<TI, BF16>, dim3((unsigned)blocks), dim3(256), 0, stream, p, log2g);
  else
    launch_kernel(lookup_kernel<TI, F32>, dim3((unsigned)blocks), dim3(256), 0, stream, p, log2g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lookup(const LookupParams &p, int table_dtype, int out_dtype,
                         hipStream_t stream) {
  if (table_dtype == kFP8) return launch_out<FP8>(p, out_dtype, stream);
  if (table_dtype == kBF16) return launch_out<BF16>(p, out_dtype, stream);
  return launch_out<F32>(p, out_dtype, stream);
}

}  // namespace dlrm
