// token_grad.hip -- gradient of the scaled token lookup:
//
//   out[r, :] = (out[r, :] or 0) + scale * sum over t with token[t] == r of grad[t, :]
//
// Tokens outside [0, rows) add nothing.  The sum of a row runs over its
// tokens in a fixed order, in float32, so equal inputs give equal bits; no
// floating-point atomic is used.
//
// Tokens are sorted by row with their positions (a stable radix sort, least
// significant digit first), so the tokens of a row are neighbours.  Then the
// sorted order is cut into chunks of equal length, whatever the rows'
// frequencies: a lane group adds up one chunk's gradient rows and stores each
// row that begins and ends inside it.  A row whose tokens cross a border
// leaves partial sums (one per chunk it touches), which the last launch adds
// in chunk order.  A token that fills a tenth of the batch is thus as well
// spread over the chip as rare ones.
//
// Digits of the sort: the key's bits are divided evenly over passes of at
// most kMaxDigit bits.  A pass is a histogram per tile of tokens and a
// scatter, in which every tile adds up the histogram for itself (bins x tiles
// counts, read from L2) instead of waiting for a scan launch.
//
// Without accumulate every row of out is written: the sort's launches occupy
// few CUs, so their grids carry further workgroups that fill out with zeros.
#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

constexpr int kMaxDigit = 10;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kItems = 4;                       // per thread
constexpr int kTile = kSortThreads * kItems;    // tokens sorted at once by a workgroup
constexpr int kMaxTiles = 512;                  // sorting workgroups (of one or more kTile)
constexpr int kFillBlocks = 512;                // zero-filling workgroups per launch
constexpr int kUnroll = 8;                      // gradient rows in flight per lane group
constexpr int kFixThreads = 512;
constexpr int kShortParts = 8;                  // chunks one lane group adds up alone

struct SortPlan {
  int passes, digit;
  int tiles, rounds;  // sorting workgroups, and the kTile tokens each takes in turn
};

SortPlan plan_sort(int64_t n, int64_t rows) {
  int bits = 1;
  while ((rows >> bits) != 0) ++bits;  // keys are 0 .. rows (rows: not there)
  SortPlan s;
  s.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  s.digit = (bits + s.passes - 1) / s.passes;
  const int64_t all = (n + kTile - 1) / kTile;
  s.rounds = (int)((all + kMaxTiles - 1) / kMaxTiles);
  s.tiles = s.rounds ? (int)((all + s.rounds - 1) / s.rounds) : 0;
  return s;
}

int lane_group_log2(int dim) {
  int g = 0;
  while ((8 << g) < dim && g < 6) ++g;
  return g;
}

// Tokens per chunk.
int chunk_tokens(int64_t n, int dim) {
  (void)n;
  (void)dim;
  return 16;
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

struct Layout {
  SortPlan s;
  int chunk;
  int64_t chunks;
  int64_t key[2], pos[2], hist, head, tail, total;  // byte offsets
};

Layout plan_layout(int64_t n, int64_t rows, int dim) {
  Layout l;
  l.s = plan_sort(n, rows);
  l.chunk = chunk_tokens(n, dim);
  l.chunks = (n + l.chunk - 1) / l.chunk;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  for (int i = 0; i < 2; ++i) {
    l.key[i] = take(n * 4);
    l.pos[i] = take(n * 4);
  }
  l.hist = take(((int64_t)4 << l.s.digit) * l.s.tiles);
  l.head = take(l.chunks * dim * 4);
  l.tail = take(l.chunks * dim * 4);
  l.total = at;
  return l;
}

// A part of out to be filled with zeros: rows [first, first + count) of
// `width` elements each (a dense out is one row of all its elements).
struct Fill {
  void *out;
  int64_t ld, first, count, width;
  int bytes;  // per element
  int blocks;
};

__device__ void fill_part(const Fill &f, int block) {
  const u32x4_t zero = {0, 0, 0, 0};
  if (f.count == 1) {  // dense: one run of bytes
    uint8_t *p = (uint8_t *)f.out + f.first * f.bytes;
    const int64_t bytes = f.width * f.bytes;
    const int64_t whole = bytes / 16;
    for (int64_t i = (int64_t)block * kSortThreads + threadIdx.x; i < whole;
         i += (int64_t)f.blocks * kSortThreads)
      put16<true>(p + i * 16, zero);
    if (block == 0)
      for (int64_t i = whole * 16 + threadIdx.x; i < bytes; i += kSortThreads) p[i] = 0;
    return;
  }
  for (int64_t r = block; r < f.count; r += f.blocks) {
    uint8_t *p = (uint8_t *)f.out + (f.first + r) * f.ld * f.bytes;
    const int64_t bytes = f.width * f.bytes;
    const int64_t whole = bytes / 16;
    for (int64_t i = threadIdx.x; i < whole; i += kSortThreads) put16<true>(p + i * 16, zero);
    for (int64_t i = whole * 16 + threadIdx.x; i < bytes; i += kSortThreads) p[i] = 0;
  }
}

struct SortPass {
  int64_t n;
  const int32_t *key_in, *pos_in;  // pos_in null: the first pass, positions are indices
  int32_t *key_out, *pos_out;
  uint32_t *hist;                  // [bin][tile]
  int32_t rows;
  int shift, digit, tiles, rounds;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass &p, int64_t i) {
  const int32_t k = p.key_in[i];
  return p.pos_in ? (uint32_t)k : (k >= 0 && k < p.rows ? (uint32_t)k : (uint32_t)p.rows);
}

// Counts of each digit in each tile of tokens.
__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(SortPass p, Fill fill) {
  extern __shared__ uint32_t lds[];
  if ((int)blockIdx.x >= p.tiles) {
    fill_part(fill, blockIdx.x - p.tiles);
    return;
  }
  const int bins = 1 << p.digit;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) lds[b] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * p.rounds * kTile;
  for (int r = 0; r < p.rounds; ++r) {
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int64_t i = first + (int64_t)r * kTile + j * kSortThreads + threadIdx.x;
      if (i < p.n) atomicAdd(&lds[(sort_key(p, i) >> p.shift) & (bins - 1)], 1u);
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    p.hist[(int64_t)b * p.tiles + blockIdx.x] = lds[b];
}

// Exclusive scan of one value per thread over the workgroup.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t *wave_sums) {
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint32_t u = __shfl_up(inc, o);
    if ((int)(threadIdx.x % kWave) >= o) inc += u;
  }
  if (threadIdx.x % kWave == kWave - 1) wave_sums[threadIdx.x / kWave] = inc;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < (int)(threadIdx.x / kWave); ++w) before += wave_sums[w];
  __syncthreads();
  return before + inc - v;
}

// Moves a tile's tokens to their places.  Equal digits keep their order:
// a wave takes 256 consecutive tokens, 64 at a time; a lane's rank among
// equal digits is what its wave has counted before plus the lower lanes with
// the same digit, found by one ballot per digit bit.
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortPass p, Fill fill) {
  extern __shared__ uint32_t lds[];
  if ((int)blockIdx.x >= p.tiles) {
    fill_part(fill, blockIdx.x - p.tiles);
    return;
  }
  const int bins = 1 << p.digit;
  __shared__ uint32_t wave_sums[kSortWaves];
  uint32_t *base = lds;                                            // [bins]
  uint16_t *count = reinterpret_cast<uint16_t *>(lds + bins);      // [waves][bins]
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  for (int b = tid; b < bins * kSortWaves / 2; b += kSortThreads)
    reinterpret_cast<uint32_t *>(count)[b] = 0;

  // first place of each digit's tokens of this tile
  const int per = bins > kSortThreads ? bins / kSortThreads : 1;
  uint32_t mine = 0;
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b < bins) {
      const uint32_t *h = p.hist + (int64_t)b * p.tiles;
      uint32_t all = 0, before = 0;
      for (int t = 0; t < p.tiles; ++t) {
        const uint32_t c = h[t];
        before += t < (int)blockIdx.x ? c : 0;
        all += c;
      }
      base[b] = mine + before;
      mine += all;
    }
  }
  const uint32_t start = block_exclusive(mine, wave_sums);
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b < bins) base[b] += start;
  }

  uint16_t *mine_count = count + wave * bins;
  for (int r = 0; r < p.rounds; ++r) {
    __syncthreads();  // counts are zero, base is this round's
    const int64_t t0 =
        ((int64_t)blockIdx.x * p.rounds + r) * kTile + wave * (kItems * kWave);
    // ranks within the wave
    uint32_t key[kItems], rank[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int64_t i = t0 + j * kWave + lane;
      key[j] = i < p.n ? sort_key(p, i) : 0;
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const bool there = t0 + j * kWave + lane < p.n;
      const uint32_t d = (key[j] >> p.shift) & (bins - 1);
      uint64_t same = __ballot(there);
      for (int b = 0; b < p.digit; ++b) {
        const uint64_t set = __ballot((d >> b) & 1);
        same &= (d >> b) & 1 ? set : ~set;
      }
      const uint32_t lower = __popcll(same & ((1ull << lane) - 1));
      const uint32_t seen = there ? mine_count[d] : 0;
      rank[j] = seen + lower;
      // the wave's LDS accesses are in order: every lane has read the count
      // before its first lane of this digit raises it
      __builtin_amdgcn_wave_barrier();
      if (there && lower == 0) mine_count[d] = (uint16_t)(seen + __popcll(same));
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // what the waves before hold of each digit
    uint32_t total[(1 << kMaxDigit) / kSortThreads];
#pragma unroll
    for (int q = 0; q < (1 << kMaxDigit) / kSortThreads; ++q) {
      const int b = tid + q * kSortThreads;
      uint32_t run = 0;
      if (b < bins) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
          const uint32_t c = count[w * bins + b];
          count[w * bins + b] = (uint16_t)run;
          run += c;
        }
      }
      total[q] = run;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int64_t i = t0 + j * kWave + lane;
      if (i < p.n) {
        const uint32_t d = (key[j] >> p.shift) & (bins - 1);
        const uint32_t to = base[d] + mine_count[d] + rank[j];
        p.key_out[to] = (int32_t)key[j];
        p.pos_out[to] = p.pos_in ? p.pos_in[i] : (int32_t)i;
      }
    }
    if (r + 1 < p.rounds) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < (1 << kMaxDigit) / kSortThreads; ++q) {
        const int b = tid + q * kSortThreads;
        if (b < bins) {
          base[b] += total[q];
#pragma unroll
          for (int w = 0; w < kSortWaves; ++w) count[w * bins + b] = 0;
        }
      }
    }
  }
}

struct ReduceParams {
  GradParams g;
  const int32_t *key, *pos;  // sorted
  float *head, *tail;        // partial sums, one row of dim each per chunk
  int64_t chunks;
  int chunk;                 // tokens per chunk
  int log2g;                 // lanes per group
  int slices;                // column slices of 8 << log2g
};

// Finishes a row: scale, earlier value, one rounding.
template <typename TO>
__device__ __forceinline__ void finish_row(const GradParams &g, int32_t row, int c,
                                           const float (&acc)[8]) {
  using SO = typename TO::S;
  SO *o = (SO *)g.out + (int64_t)row * g.ld_out;
  float v[8];
  if (g.accumulate) {
    load_chunk<TO>(o, c, g.dim, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(g.scale, acc[e], v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = g.scale * acc[e];
  }
  store_chunk<TO>(o, c, g.dim, v);
}

template <typename TG, typename TO>
__global__ __launch_bounds__(256) void grad_reduce_kernel(ReduceParams p) {
  using SG = typename TG::S;
  const int G = 1 << p.log2g;
  const int lane = threadIdx.x & (G - 1);
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> p.log2g;
  const int64_t chunk = item / p.slices;
  if (chunk >= p.chunks) return;
  const int c = ((int)(item - chunk * p.slices) * G + lane) * 8;
  if (c >= p.g.dim) return;
  const int32_t rows = (int32_t)p.g.rows;
  const int64_t s0 = chunk * p.chunk;
  const int64_t s1 = s0 + p.chunk < p.g.n ? s0 + p.chunk : p.g.n;
  const int32_t before = s0 > 0 ? p.key[s0 - 1] : -1;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  bool fresh = true;  // the running row began in this chunk
  for (int64_t s = s0; s < s1; s += kUnroll) {
    int32_t key[kUnroll + 1];
    float v[kUnroll][8];
#pragma unroll
    for (int j = 0; j <= kUnroll; ++j) key[j] = s + j < p.g.n ? p.key[s + j] : rows;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      // (positions of the chunk only: a chunk is a multiple of kUnroll)
      if (key[j] < rows) {
        load_chunk<TG>((const SG *)p.g.grad + (int64_t)p.pos[s + j] * p.g.ld_grad, c, p.g.dim,
                       v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
      }
    }
    if (s == s0) fresh = before != key[0];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (key[j] >= rows) return;  // only tokens outside the table follow
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[j][e];
      const bool more = key[j + 1] == key[j];
      const bool border = s + j + 1 == s1;
      if (!more || border) {
        if (!fresh)
          store_chunk<F32>(p.head + chunk * p.g.dim, c, p.g.dim, acc);
        else if (more)
          store_chunk<F32>(p.tail + chunk * p.g.dim, c, p.g.dim, acc);
        else
          finish_row<TO>(p.g, key[j], c, acc);
        fresh = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
      }
    }
  }
}

// Whether a row's tokens begin in `chunk` and go on in the next one.
__device__ __forceinline__ bool crosses(const ReduceParams &p, int64_t chunk, int32_t &key) {
  const int64_t s1 = (chunk + 1) * p.chunk;
  if (s1 >= p.g.n) return false;
  key = p.key[s1 - 1];
  if (key >= p.g.rows || p.key[s1] != key) return false;
  const int64_t s0 = chunk * p.chunk;
  return p.key[s0] != key || s0 == 0 || p.key[s0 - 1] != key;
}

// How many chunks after `chunk` a crossing row reaches, counted up to limit.
__device__ __forceinline__ int parts_after(const ReduceParams &p, int64_t chunk, int32_t key,
                                           int limit) {
  int n = 0;
  for (int k = 1; k <= limit; ++k) {
    const int64_t s = (chunk + k) * p.chunk;
    n += s < p.g.n && p.key[s] == key ? 1 : 0;
  }
  return n;
}

// Adds the partial sums of rows that cross chunks.  A workgroup looks at as
// many chunks as it has lane groups.  A row of few chunks is added by its
// lane group; a longer one by the whole workgroup, each lane group a run of
// its partials, the runs' sums in order through LDS.
template <typename TO>
__global__ __launch_bounds__(kFixThreads) void grad_fix_kernel(ReduceParams p) {
  const int G = 1 << p.log2g, NG = kFixThreads >> p.log2g;
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x >> p.log2g;
  const int slice = blockIdx.y;
  const int c = (slice * G + lane) * 8;
  const bool live = c < p.g.dim;
  const int64_t first = (int64_t)blockIdx.x * NG;
  __shared__ int nlong;
  __shared__ int64_t longs[kFixThreads];
  __shared__ float sums[kFixThreads][8];
  if (threadIdx.x == 0) nlong = 0;
  __syncthreads();
  {
    const int64_t chunk = first + group;
    int32_t key = 0;
    if (chunk < p.chunks && crosses(p, chunk, key)) {
      const int n = parts_after(p, chunk, key, kShortParts + 1);
      if (n <= kShortParts) {
        if (live) {
          float acc[8], v[kShortParts][8];
          load_chunk<F32>(p.tail + chunk * p.g.dim, c, p.g.dim, acc);
#pragma unroll
          for (int k = 0; k < kShortParts; ++k)
            if (k < n) load_chunk<F32>(p.head + (chunk + 1 + k) * p.g.dim, c, p.g.dim, v[k]);
#pragma unroll
          for (int k = 0; k < kShortParts; ++k)
            if (k < n)
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[e] += v[k][e];
          finish_row<TO>(p.g, key, c, acc);
        }
      } else if (lane == 0) {
        longs[atomicAdd(&nlong, 1)] = chunk;
      }
    }
  }
  __syncthreads();
  const int todo = nlong;
  for (int w = 0; w < todo; ++w) {
    const int64_t chunk = longs[w];
    const int32_t key = p.key[(chunk + 1) * p.chunk - 1];
    int64_t n = 0;  // chunks after this one that the row reaches
    for (;;) {
      const int64_t s = (chunk + 1 + n + threadIdx.x) * p.chunk;
      const int got = __syncthreads_count(s < p.g.n && p.key[s] == key);
      n += got;
      if (got < kFixThreads) break;
    }
    // partial 0 is the tail, partial k the head of chunk + k
    const int64_t per = (n + 1 + NG - 1) / NG;
    const int64_t k0 = group * per, k1 = k0 + per < n + 1 ? k0 + per : n + 1;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    if (live) {
      for (int64_t k = k0; k < k1; k += kUnroll) {
        float v[kUnroll][8];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          if (k + j < k1) {
            const float *src = k + j == 0 ? p.tail + chunk * p.g.dim
                                          : p.head + (chunk + k + j) * p.g.dim;
            load_chunk<F32>(src, c, p.g.dim, v[j]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
          }
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[j][e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = acc[e];
    __syncthreads();
    if (group == 0 && live) {
      for (int q = 1; q < NG; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += sums[q * G + lane][e];
      finish_row<TO>(p.g, key, c, acc);
    }
    __syncthreads();
  }
}

Fill part_of(const GradParams &g, int out_bytes, int part, int parts) {
  Fill f{};
  f.out = g.out;
  f.ld = g.ld_out;
  f.bytes = out_bytes;
  if (g.accumulate) return f;
  if (g.ld_out == g.dim) {
    const int64_t all = g.rows * g.dim;
    const int64_t a = all * part / parts / 8 * 8;
    const int64_t b = part + 1 == parts ? all : all * (part + 1) / parts / 8 * 8;
    f.first = a;
    f.count = 1;
    f.width = b - a;
    const int64_t want = (f.width * out_bytes / 16 + kSortThreads - 1) / kSortThreads;
    f.blocks = (int)(want < 1 ? 1 : want < kFillBlocks ? want : kFillBlocks);
  } else {
    const int64_t a = g.rows * part / parts, b = g.rows * (part + 1) / parts;
    f.first = a;
    f.count = b - a;
    f.width = g.dim;
    f.blocks = (int)(f.count < kFillBlocks ? f.count : kFillBlocks);
    if (f.count == 1) f.first = a * g.ld_out;  // a single row is one run too
  }
  return f;
}

template <typename TG, typename TO>
hipError_t launch_typed(const GradParams &g, void *ws, hipStream_t stream) {
  const int ob = (int)sizeof(typename TO::S);
  uint8_t *w = (uint8_t *)ws;
  const Layout l = plan_layout(g.n, g.rows, g.dim);
  const int parts = g.n > 0 ? 2 * l.s.passes : 1;
  SortPass sp{};
  sp.n = g.n;
  sp.rows = (int32_t)g.rows;
  sp.digit = l.s.digit;
  sp.tiles = l.s.tiles;
  sp.rounds = l.s.rounds;
  sp.hist = (uint32_t *)(w + l.hist);
  sp.key_in = g.token;
  hipError_t e;
  if (g.n == 0) {  // tiles is 0: the launch only fills
    const Fill f = part_of(g, ob, 0, 1);
    if (f.blocks > 0)
      launch_kernel(sort_hist_kernel, dim3(f.blocks), dim3(kSortThreads), 0, stream, sp, f);
    return hipGetLastError();
  }
  const size_t bins = (size_t)1 << l.s.digit;
  for (int pass = 0; pass < l.s.passes; ++pass) {
    sp.shift = pass * l.s.digit;
    sp.key_out = (int32_t *)(w + l.key[pass & 1]);
    sp.pos_out = (int32_t *)(w + l.pos[pass & 1]);
    Fill f = part_of(g, ob, 2 * pass, parts);
    launch_kernel(sort_hist_kernel, dim3(sp.tiles + f.blocks), dim3(kSortThreads), bins * 4,
                  stream, sp, f);
    f = part_of(g, ob, 2 * pass + 1, parts);
    launch_kernel(sort_scatter_kernel, dim3(sp.tiles + f.blocks), dim3(kSortThreads),
                  bins * (4 + 2 * kSortWaves), stream, sp, f);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    sp.key_in = sp.key_out;
    sp.pos_in = sp.pos_out;
  }
  ReduceParams rp{};
  rp.g = g;
  rp.key = sp.key_in;
  rp.pos = sp.pos_in;
  rp.head = (float *)(w + l.head);
  rp.tail = (float *)(w + l.tail);
  rp.chunks = l.chunks;
  rp.chunk = l.chunk;
  rp.log2g = lane_group_log2(g.dim);
  rp.slices = (g.dim + (8 << rp.log2g) - 1) / (8 << rp.log2g);
  const int64_t lanes = (rp.chunks * rp.slices) << rp.log2g;
  launch_kernel(grad_reduce_kernel<TG, TO>, dim3((unsigned)((lanes + 255) / 256)), dim3(256), 0,
                stream, rp);
  const int ng = kFixThreads >> rp.log2g;
  launch_kernel(grad_fix_kernel<TO>, dim3((unsigned)((rp.chunks + ng - 1) / ng), rp.slices),
                dim3(kFixThreads), 0, stream, rp);
  return hipGetLastError();
}

}  // namespace

size_t lookup_grad_workspace(int64_t n, int64_t rows, int dim) {
  return n > 0 ? (size_t)plan_layout(n, rows, dim).total : 0;
}

hipError_t launch_lookup_grad(const GradParams &g, int grad_dtype, int out_dtype, void *ws,
                              hipStream_t stream) {
  if (grad_dtype == kBF16)
    return out_dtype == kBF16 ? launch_typed<BF16, BF16>(g, ws, stream)
                              : launch_typed<BF16, F32>(g, ws, stream);
  return out_dtype == kBF16 ? launch_typed<F32, BF16>(g, ws, stream)
                            : launch_typed<F32, F32>(g, ws, stream);
}

}  // namespace dlrm
