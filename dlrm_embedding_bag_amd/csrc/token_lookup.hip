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
// memory.  One row for each group: the chain of two memory round trips (token,
// then row) is hidden by the many groups of a CU, better than by several rows
// in a group's registers (4 million rows of 16: 43 us, 58 with two rows, 86
// with four).  Outputs are streamed past the caches (nontemporal stores), so
// that what the caches hold is rows that other tokens will ask for: 262144
// tokens x 1024 bfloat16 of a Zipf batch take 98 us, 163 without.  That is
// 5.9 TB/s of outputs, tokens and distinct rows; the stores bound it.
#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

constexpr int64_t kMaxBlocks = 1 << 22;  // a launch holds fewer than 2^32 threads

template <typename TI, typename TO>
__global__ __launch_bounds__(256) void lookup_kernel(LookupParams p, int log2g) {
  using SI = typename TI::S;
  using SO = typename TO::S;
  constexpr int V = 16 / (int)sizeof(SO);  // elements of a chunk
  const int G = 1 << log2g;
  const int lane = threadIdx.x & (G - 1);
  const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> log2g;
  for (int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> log2g; t < p.tokens;
       t += step) {
    const int32_t tok = p.token[t];
    const bool there = tok >= 0 && tok < p.rows;
    const SI *row = (const SI *)p.table + (there ? (int64_t)tok * p.ld_table : 0);
    SO *out = (SO *)p.out + t * p.ld_out;
    for (int c = lane * V; c < p.dim; c += G * V) {
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 0.0f;
      if (there) load_chunk<TI>(row, c, p.dim, v);
      // a row that is not there is zero whatever the scale is
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = there ? v[e] * p.scale : 0.0f;
      store_chunk<TO, true>(out, c, p.dim, v);
    }
  }
}

template <typename TI, typename TO>
hipError_t launch_typed(const LookupParams &p, hipStream_t stream) {
  constexpr int V = 16 / (int)sizeof(typename TO::S);
  int log2g = 0;
  while ((V << log2g) < p.dim && log2g < 6) ++log2g;
  const int64_t want = ((p.tokens << log2g) + 255) / 256;
  const int64_t blocks = want < kMaxBlocks ? want : kMaxBlocks;
  launch_kernel(lookup_kernel<TI, TO>, dim3((unsigned)blocks), dim3(256), 0, stream, p, log2g);
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
