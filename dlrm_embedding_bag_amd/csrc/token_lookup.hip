// token_lookup.hip -- embedding lookup of single tokens with a scale:
//
//   out[t, :] = scale * table[token[t], :]     (zeros outside [0, rows))
//
// float32, bfloat16 or FP8 E4M3 rows, the product in float32, rounded once to
// the output type.  The kernel moves bytes: it is bound by the stores and by
// the distinct rows' reads.
//
// A row belongs to a group of G lanes (a power of two, up to a wave), each
// taking chunks whose output is 16 bytes, so that a group's store is one run of
// memory.  Outputs are streamed past the caches (nontemporal stores), so that
// what the caches hold is rows that other tokens will ask for: 262144 tokens x
// 1024 bfloat16 of a Zipf batch, tables and tokens new each time, take 107 us a
// call (110 in a kernel trace), 5.7 TB/s of outputs, tokens and distinct rows;
// the memory bounds it.  (With ordinary stores 164, beside 115 in that run.)
// A row that ends inside a chunk pays for the rounding of its lanes to a power
// of two and for the last chunk, element by element: 2000000 tokens x 64 float32
// take 131 us, x 65 175; bfloat16 x 32 37, x 33 62, x 64 62.
#include <type_traits>

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

constexpr int64_t kMaxBlocks = 1 << 22;  // a launch holds fewer than 2^32 threads

template <typename TI, typename TO, int ROWS>
__global__ __launch_bounds__(256) void lookup_kernel(LookupParams p, int log2g) {
  using SI = typename TI::S;
  using SO = typename TO::S;
  constexpr int V = 16 / (int)sizeof(SO);  // elements of a chunk
  const int G = 1 << log2g;
  const int lane = threadIdx.x & (G - 1);
  const int64_t group = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> log2g;
  const int64_t step = (((int64_t)gridDim.x * blockDim.x) >> log2g) * ROWS;
  for (int64_t t = group * ROWS; t < p.tokens; t += step) {
    int32_t tok[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) tok[r] = t + r < p.tokens ? p.token[t + r] : -1;
    for (int c = lane * V; c < p.dim; c += G * V) {
      float v[ROWS][V];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[r][e] = 0.0f;
        if (tok[r] >= 0 && tok[r] < p.rows)
          load_chunk<TI>((const SI *)p.table + (int64_t)tok[r] * p.ld_table, c, p.dim, v[r]);
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        // a row that is not there is zero whatever the scale is
        const bool there = tok[r] >= 0 && tok[r] < p.rows;
#pragma unroll
        for (int e = 0; e < V; ++e) v[r][e] = there ? v[r][e] * p.scale : 0.0f;
        if (t + r < p.tokens) store_chunk<TO, true>((SO *)p.out + (t + r) * p.ld_out, c, p.dim, v[r]);
      }
    }
  }
}

template <typename TI, typename TO>
hipError_t launch_typed(const LookupParams &p, hipStream_t stream) {
  constexpr int V = 16 / (int)sizeof(typename TO::S);
  int log2g = 0;
  while ((V << log2g) < p.dim && log2g < 6) ++log2g;
  // Rows of a group in flight.  The chain of two memory round trips (token, then
  // row) is hidden by the other groups of a CU where there are many; long rows
  // fill it with few (262144 x 1024: 136 us with one, 120 with two, 115 with
  // four), short ones want few registers (4 million x 16: 43, 58, 88 us), and
  // few tokens want every CU (1000 x 512: 2.8, 3.0, 3.4 us).
  auto launch = [&](auto rows) {
    constexpr int ROWS = decltype(rows)::value;
    const int64_t want = (((p.tokens + ROWS - 1) / ROWS << log2g) + 255) / 256;
    const int64_t blocks = want < kMaxBlocks ? want : kMaxBlocks;
    launch_kernel(lookup_kernel<TI, TO, ROWS>, dim3((unsigned)blocks), dim3(256), 0, stream, p,
                  log2g);
  };
  if (log2g < 3 || p.tokens << log2g < 1 << 20)
    launch(std::integral_constant<int, 1>());
  else if (log2g < 6)
    launch(std::integral_constant<int, 2>());
  else
    launch(std::integral_constant<int, 4>());
  return hipGetLastError();
}

template <typename TI>
hipError_t launch_out(const LookupParams &p, int out_dtype, hipStream_t stream) {
  return out_dtype == kBF16 ? launch_typed<TI, BF16>(p, stream) : launch_typed<TI, F32>(p, stream);
}

}  // namespace

hipError_t launch_lookup(const LookupParams &p, int table_dtype, int out_dtype,
                         hipStream_t stream) {
  if (table_dtype == kFP8) return launch_out<FP8>(p, out_dtype, stream);
  if (table_dtype == kBF16) return launch_out<BF16>(p, out_dtype, stream);
  return launch_out<F32>(p, out_dtype, stream);
}

}  // namespace dlrm
