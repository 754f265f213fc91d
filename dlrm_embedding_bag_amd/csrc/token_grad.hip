// token_grad.hip -- gradient of the scaled token lookup:
//
//   out[r, :] = (out[r, :] or 0) + scale * sum over t with token[t] == r of grad[t, :]
//
// Tokens outside [0, rows) add nothing.  The sum of a row runs over its
// tokens in an order that the tokens alone decide, in float32, so equal inputs
// give equal bits; no floating-point atomic is used.
//
// Tokens are sorted by row, equal ones by position, so the tokens of a row are
// neighbours; then the sorted order is cut into equal parts, whatever the
// rows' frequencies, so that a token that fills a tenth of the batch is as
// well spread over the chip as rare ones.
//
// Up to kTile tokens, one launch does everything: each of its workgroups
// sorts all tokens in its registers and LDS (none waits for another) and adds
// up its share of the sorted order; others write zeros to the rows that no
// token names.
//
// Beyond, four launches (more where one merge does not reach all tokens):
//   tile_sort   tiles of kTile tokens, each sorted by one workgroup
//   merge       a token's place among the sorted runs is its place in its own
//               run plus, for each other run, a binary search: thousands of
//               independent searches that stay in the caches, in one launch
//               where a radix sort takes two for each digit
//   reduce      workgroups add up equal parts of the sorted order; a row that
//               crosses a border leaves partial sums
//   fix         adds those in order
// Without accumulate every row of out is written: the sort's launches occupy
// few CUs, so their grids carry further workgroups that fill out with zeros.
//
// Kernel times of Zipf batches (us):    sort  merge  reduce  fix
//   40960 x 64 f32 into 1M rows            7     11      8     5   launches and
//     the searches' chain bound it; its 18 MB would take 4
//   65536 x 1024 bf16, 100000 rows f32    34     41     44     6   400 MB of
//     zeros behind the sort (6 TB/s), then 134 MB of gradients and 80 MB of
//     rows (4.9 TB/s): memory bounds it, but for the merge's 13 us
//   500000 x 16 bf16 into 500000 rows      8  2 x 66     20     9   beyond 65536
//     tokens the merges bound it, n (fan - 1) log2(run) steps of search each;
//     its 29 MB would take 6
//   160 x 16 (one launch): 5; 1000 x 64: 11
#include <type_traits>

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

namespace {

constexpr int kThreads = 512;                 // of a sorting workgroup
constexpr int kWaves = kThreads / kWave;
constexpr int kFew = 2;                       // tokens of a thread that sorts few,
constexpr int kMany = 4;                      // and many
constexpr int kTile = kMany * kThreads;       // tokens that one workgroup sorts (2048 take 7 us,
                                              // 4096 in twice the threads 14)
constexpr int kOneMerge = 32;                 // runs merged at once where that ends it,
constexpr int kMaxFan = 16;                   // and else
constexpr int kMergeWaves = 8;
constexpr int kMergeThreads = kMergeWaves * kWave;
constexpr int kSearches = 4;                  // binary searches of a thread in flight
constexpr int kMergeBlocks = 1 << 16;         // merging workgroups, at most (the chip holds 1024)
constexpr int kFillBlocks = 1 << 16;          // zero-filling workgroups per launch, at most
constexpr int kReduceThreads = 256;
constexpr int kMaxPer = 8;                    // tokens that a lane group adds up alone
constexpr int kMaxPart = 256 * kMaxPer;       // tokens of a part
constexpr int kFixThreads = 256;
constexpr int kUnroll = 8;                    // partial sums of a lane group in flight
constexpr int64_t kMaxBlocks = 1 << 22;       // a launch holds fewer than 2^32 threads

// ------------------------------------------------------------------ sort --

// The lower of two values, or the upper.
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b, bool low) {
  const uint32_t x = a < b ? a : b, y = a < b ? b : a;
  return low ? x : y;
}
__device__ __forceinline__ uint64_t pick(uint64_t a, uint64_t b, bool low) {
  return (a < b) == low ? a : b;
}

// Puts v[a], v[b] of a thread in order.
template <typename K>
__device__ __forceinline__ void in_order(K &a, K &b) {
  const K x = a < b ? a : b, y = a < b ? b : a;
  a = x;
  b = y;
}

// Steps at distances within a thread: H, H / 2, ..., 1.
template <int H, typename K, int E>
__device__ __forceinline__ void thread_steps(K (&v)[E]) {
  if constexpr (H > 0) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((e & H) == 0) in_order(v[e], v[e + H]);
    thread_steps<H / 2>(v);
  }
}

// Sorts the values of a thread.
template <int N, typename K, int E>
__device__ __forceinline__ void thread_levels(K (&v)[E]) {
  if constexpr (N <= E) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((e & (N / 2)) == 0) in_order(v[e], v[e ^ (N - 1)]);
    thread_steps<N / 4>(v);
    thread_levels<N * 2>(v);
  }
}

// Steps at a distance of LANES lanes, of LANES / 2, and so on down to 1 value.
template <int LANES, typename K, int E>
__device__ __forceinline__ void close_steps(K (&v)[E]) {
  if constexpr (LANES > 0) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      v[e] = pick(v[e], lane_xor<LANES>(v[e]), (threadIdx.x & LANES) == 0);
    close_steps<LANES / 2>(v);
  } else {
    thread_steps<E / 2>(v);
  }
}

// Merges sorted runs of LANES / 2 lanes, and so on up to a whole wave.
template <int LANES, typename K, int E>
__device__ __forceinline__ void wave_levels(K (&v)[E]) {
  K o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = lane_xor<LANES - 1>(v[E - 1 - e]);
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = pick(v[e], o[e], (threadIdx.x & (LANES / 2)) == 0);
  close_steps<LANES / 4>(v);
  if constexpr (LANES < kWave) wave_levels<LANES * 2>(v);
}

// Sort of P values (a power of two, at least 64 E) by the workgroup: thread t
// holds values [t E, t E + E) before and after.  A sorting network: a level
// joins pairs of sorted runs by comparing each value with its mirror image in
// the pair, then at half the distance and so on, the lower value always to the
// lower place.  (With that order a step is a move between lanes, a minimum, a
// maximum and a choice by a constant lane mask; instructions bound it.)  The
// more values a thread holds, the more of the steps lie within a thread, where
// they take no move and no choice.  Longer distances than a wave go through
// two LDS buffers in turn, one barrier each.  `lds` holds 2 P values.
template <typename K, int E>
__device__ void block_sort(K (&v)[E], K *lds, int P) {
  const int first = threadIdx.x * E;
  const bool there = first < P;
  if (there) {
    thread_levels<2>(v);
    wave_levels<2>(v);
  }
  int buf = 0;
  for (int k = 2 * kWave * E; k <= P; k <<= 1) {
    for (int half = k >> 1; half >= kWave * E; half >>= 1) {
      const bool mirror = 2 * half == k;
      K *b = lds + buf * P;
      buf ^= 1;
      if (there) {
#pragma unroll
        for (int e = 0; e < E; ++e) b[first + e] = v[e];
      }
      __syncthreads();
      if (there) {  // a thread's partners are the values of one thread
        const K *q = b + (first ^ (mirror ? k - E : half));
        K o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = q[e];
        const bool low = (first & half) == 0;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = pick(v[e], mirror ? o[E - 1 - e] : o[e], low);
      }
    }
    if (there) close_steps<kWave / 2>(v);
  }
}

// What is sorted: the row in the upper bits, the token's index within the
// tile in the lower ones.  32 bits where both fit, else 64.
template <typename K, int E>
__host__ __device__ constexpr int index_bits() {
  return sizeof(K) == 8 ? 32 : (E == kFew ? 10 : 11);
}

template <int E>
constexpr int64_t kRows32 = (int64_t)1 << (32 - index_bits<uint32_t, E>());  // table rows below it

__device__ __forceinline__ uint32_t row_of(int32_t token, int64_t rows) {
  return token >= 0 && token < rows ? (uint32_t)token : (uint32_t)rows;  // rows: not there
}

// Values [first, first + E) of the tile of n tokens at `token`; all ones past
// its end.
template <typename K, int E>
__device__ __forceinline__ void load_tile(const int32_t *token, int n, int64_t rows, K (&v)[E]) {
  const int first = threadIdx.x * E;
  int32_t t[E];
#pragma unroll
  for (int e = 0; e < E; ++e) t[e] = first + e < n ? token[first + e] : -1;
#pragma unroll
  for (int e = 0; e < E; ++e)
    v[e] = first + e < n
               ? (K)row_of(t[e], rows) << index_bits<K, E>() | (K)(uint32_t)(first + e)
               : ~(K)0;
}

// ------------------------------------------------------------------ fill --

// A part of out to be filled with zeros: rows [first, first + count) of
// `width` elements each (a dense out is one row of all its elements).
struct Fill {
  void *out;
  int64_t ld, first, count, width;
  int bytes;  // per element
  int blocks;
};

// `t` of `threads` threads write zeros to a run of bytes, 16 at a time.
__device__ __forceinline__ void zero_run(uint8_t *p, int64_t bytes, int64_t t, int64_t threads) {
  const u32x4_t zero = {0, 0, 0, 0};
  const int64_t whole = bytes / 16;
  for (int64_t i = t; i < whole; i += threads) put16<true>(p + i * 16, zero);
  for (int64_t i = whole * 16 + t; i < bytes; i += threads) p[i] = 0;
}

__device__ void fill_part(const Fill &f, int block) {
  if (f.count == 1) {  // dense: one run of bytes
    zero_run((uint8_t *)f.out + f.first * f.bytes, f.width * f.bytes,
             (int64_t)block * blockDim.x + threadIdx.x, (int64_t)f.blocks * blockDim.x);
    return;
  }
  for (int64_t r = block; r < f.count; r += f.blocks)
    zero_run((uint8_t *)f.out + (f.first + r) * f.ld * f.bytes, f.width * f.bytes, threadIdx.x,
             blockDim.x);
}

// ---------------------------------------------------------------- reduce --

// Finishes a row: scale, earlier value, one rounding.
template <typename TO>
__device__ __forceinline__ void finish_row(const GradParams &g, uint32_t row, int c,
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

// A lane group: the lanes that hold one row of a column slice, 8 elements each.
struct Lanes {
  int group, groups;  // of the workgroup
  int log2g;          // log2 of its lanes
  int c;              // first column of this lane
  bool live;          // c < dim
};

__device__ __forceinline__ Lanes lanes_of(int log2g, int64_t slice, int dim) {
  const int G = 1 << log2g;
  Lanes l;
  l.log2g = log2g;
  l.group = threadIdx.x >> log2g;
  l.groups = blockDim.x >> log2g;
  const int64_t c = (slice * G + (threadIdx.x & (G - 1))) * 8;
  l.live = c < dim;
  l.c = l.live ? (int)c : 0;
  return l;
}

// Adds up the sorted tokens [t0, t1) by the workgroup, PER (or fewer at the
// end) for each lane group.  A row that lies in one group's tokens is finished
// there.  What a group holds of a row that began before it, its head, is
// added to the group in which the row begins: within a wave by a scan over its
// groups (a frequent row's tokens fill many groups, and a step by step walk
// over them took longer than their loads), from wave to wave through `heads`
// in LDS (two arrays of one float4 per thread).
//   key(i), pos(i)   row and position of sorted token i
//   open             the row of t0 began before it: group 0 takes it up from
//                    what begin(acc) gives
//   goes_on          the row of t1 - 1 goes on after it: end(row, acc) takes its
//                    sum so far
//   done(row, acc)   takes a finished row
template <typename TG, int PER, typename Key, typename Pos, typename Begin, typename End,
          typename Done>
__device__ __forceinline__ void reduce_tokens(const GradParams &g, const Lanes &l, int t0, int t1,
                                              bool open, bool goes_on, f32x4_t *heads,
                                              Key key, Pos pos, Begin begin, End end, Done done) {
  using SG = typename TG::S;
  const int a = t0 + l.group * PER;
  const int b = a + PER < t1 ? a + PER : t1;
  float acc[8], head[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = head[e] = 0.0f;
  bool tail = false;  // acc holds a row that begins here and goes on
  bool pass = false;  // head holds all tokens of the group, and their row goes on
  if (l.live && a < b) {
    Chunk<TG> v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (a + j < b) v[j].load((const SG *)g.grad + (int64_t)pos(a + j) * g.ld_grad, l.c, g.dim);
    bool fresh = a == t0 ? !open : key(a - 1) != key(a);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (a + j < b) {
        const uint32_t row = key(a + j);
        const bool more = a + j + 1 < t1 ? key(a + j + 1) == row : goes_on;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += v[j].at(e);
        if (!more || a + j + 1 == b) {
          if (!fresh) {
#pragma unroll
            for (int e = 0; e < 8; ++e) head[e] = acc[e];
            pass = more;
          } else if (more) {
            tail = true;
          } else {
            done(row, acc);
          }
          fresh = true;
          if (!tail) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
          }
        }
      }
    }
  }
  // head: the group's and, where its row goes on, those of the wave's groups
  // after it, as far as the row reaches
  const int G = 1 << l.log2g, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  for (int d = G; d < kWave; d <<= 1) {
    const bool next = __shfl_down((int)pass, d);
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __shfl_down(head[e], d);
    if (pass && lane + d < kWave) {
#pragma unroll
      for (int e = 0; e < 8; ++e) head[e] += o[e];
      pass = next;
    }
  }
  if (G < kWave) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_down(head[e], G);
      if (tail && lane + G < kWave) acc[e] += o;
    }
  }
  f32x4_t *head_lo = heads, *head_hi = heads + blockDim.x;
  if (lane < G) {
    head_lo[wave * G + lane] = f32x4_t{head[0], head[1], head[2], head[3]};
    head_hi[wave * G + lane] = f32x4_t{head[4], head[5], head[6], head[7]};
  }
  __syncthreads();
  // adds the heads of the waves after this one that the row reaches
  auto walk = [&](uint32_t row) {
    const int stride = (kWave >> l.log2g) * PER;
    int w = wave + 1;
    for (int s = t0 + w * stride; s < t1 && key(s) == row; s += stride, ++w) {
      const f32x4_t lo = head_lo[w * G + lane % G], hi = head_hi[w * G + lane % G];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[e] += lo[e];
        acc[4 + e] += hi[e];
      }
    }
    if (goes_on && key(t1 - 1) == row)
      end(row, acc);
    else
      done(row, acc);
  };
  if (tail) walk(key(b - 1));
  if (open && l.group == 0 && l.live && t0 < t1) {
    begin(acc);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += head[e];
    walk(key(t0));
  }
}

// ------------------------------------------------------------ one launch --

struct SmallParams {
  GradParams g;
  int P;         // power of two that holds the tokens
  int segments;  // parts of the sorted order
  int slices;    // column slices of 8 << log2g
  int log2g;
};

// Zeros for those of rows [r0, r1) that no token names, by one workgroup: a
// bitmap of the rows in LDS (kBitmap bits), one mark for each token.
constexpr int kBitmap = 1 << 16;
template <int BYTES>
__device__ void fill_unnamed(const GradParams &g, int64_t r0, int64_t r1, uint32_t *bits) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int64_t row_bytes = (int64_t)g.dim * BYTES, ld_bytes = g.ld_out * BYTES;
  int share = 0;  // log2 of the lanes that share a row
  while (share < 6 && (16 << share) < row_bytes) ++share;
  for (int64_t q0 = r0; q0 < r1; q0 += kBitmap) {
    const int count = r1 - q0 < kBitmap ? (int)(r1 - q0) : kBitmap;
    for (int i = threadIdx.x; i < (count + 31) / 32; i += kThreads) bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < (int)g.n; i += kThreads) {
      const int64_t r = g.token[i] - q0;  // (a token outside the table is outside [q0, r1))
      if (r >= 0 && r < count) atomicOr(&bits[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    const int each = (count + kWaves - 1) / kWaves < kWave ? (count + kWaves - 1) / kWaves : kWave;
    for (int r = wave * each; r < count; r += kWaves * each) {
      const int rows = count - r < each ? count - r : each;
      const bool named = lane < rows && (bits[(r + lane) >> 5] >> ((r + lane) & 31) & 1);
      const uint64_t mask = __ballot(named);
      uint8_t *o = (uint8_t *)g.out + (q0 + r) * ld_bytes;
      if (mask == 0 && ld_bytes == row_bytes) {
        zero_run(o, rows * row_bytes, lane, kWave);
      } else {
        for (int q = lane >> share; q < rows; q += kWave >> share)
          if (!((mask >> q) & 1))
            zero_run(o + q * ld_bytes, row_bytes, lane & ((1 << share) - 1), 1 << share);
      }
    }
    __syncthreads();
  }
}

template <typename TG, typename TO, typename K, int E>
__global__ __launch_bounds__(kThreads) void small_kernel(SmallParams p) {
  constexpr int B = index_bits<K, E>();
  __shared__ K sorted[2 * kThreads * E];
  __shared__ f32x4_t heads[2 * kThreads];
  __shared__ f32x4_t carry[2][2][kWave];  // the open row's sum, by round parity
  const GradParams &g = p.g;
  const int n = (int)g.n;
  if ((int)blockIdx.x >= p.segments * p.slices) {
    const int blocks = gridDim.x - p.segments * p.slices;
    const int64_t b = blockIdx.x - p.segments * p.slices;
    fill_unnamed<sizeof(typename TO::S)>(g, g.rows * b / blocks, g.rows * (b + 1) / blocks,
                                         (uint32_t *)sorted);
    return;
  }
  K v[E];
  load_tile<K, E>(g.token, n, g.rows, v);
  int nv = 0;  // tokens in the table
#pragma unroll
  for (int e = 0; e < E; ++e)
    nv += __syncthreads_count((uint64_t)(v[e] >> B) < (uint64_t)g.rows ? 1 : 0);
  block_sort<K, E>(v, sorted, p.P);
  __syncthreads();
  if ((int)threadIdx.x * E < p.P) {
#pragma unroll
    for (int e = 0; e < E; ++e) sorted[threadIdx.x * E + e] = v[e];
  }
  __syncthreads();
  auto key = [&](int i) { return (uint32_t)(sorted[i] >> B); };
  auto pos = [&](int i) { return (uint32_t)sorted[i] & (uint32_t)(((uint64_t)1 << B) - 1); };
  // the first sorted token whose row is not below `row`
  auto place = [&](uint32_t row) {
    int at = 0;
    for (int s = p.P >> 1; s > 0; s >>= 1)
      if (at + s <= nv && key(at + s - 1) < row) at += s;
    return at + (at < nv && key(at) < row ? 1 : 0);
  };

  const Lanes l = lanes_of(p.log2g, blockIdx.x % p.slices, g.dim);
  const int seg = blockIdx.x / p.slices;
  const int len = (nv + p.segments - 1) / p.segments;
  // a segment owns the rows that begin in it, to their last token
  auto border = [&](int s) {
    if (s >= nv) return nv;
    if (s > 0 && key(s - 1) == key(s)) return place(key(s) + 1);
    return s;
  };
  const int start = border(seg * len), stop = border((seg + 1) * len);
  const int lane = threadIdx.x & ((1 << p.log2g) - 1);
  auto add_up = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    int round = 0;
    for (int t0 = start; t0 < stop; t0 += l.groups * PER, round ^= 1) {
      const int t1 = t0 + l.groups * PER < stop ? t0 + l.groups * PER : stop;
      reduce_tokens<TG, PER>(
          g, l, t0, t1, t0 > start && key(t0 - 1) == key(t0),
          t1 < stop && key(t1 - 1) == key(t1), heads, key, pos,
          [&](float (&acc)[8]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[e] = carry[round][0][lane][e];
              acc[4 + e] = carry[round][1][lane][e];
            }
          },
          [&](uint32_t, const float (&acc)[8]) {
            carry[round ^ 1][0][lane] = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
            carry[round ^ 1][1][lane] = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
          },
          [&](uint32_t row, const float (&acc)[8]) { finish_row<TO>(g, row, l.c, acc); });
      __syncthreads();  // heads are read before the next round writes them
    }
  };
  // a token for each lane group where that is one round, else eight
  if (stop - start <= l.groups)
    add_up(std::integral_constant<int, 1>());
  else
    add_up(std::integral_constant<int, kMaxPer>());
}

// --------------------------------------------------------- sorting tokens --

template <typename K>
__global__ __launch_bounds__(kThreads) void tile_sort_kernel(const int32_t *token, int64_t n,
                                                             int64_t rows, int tiles, int32_t *key,
                                                             int32_t *pos, Fill fill) {
  constexpr int E = kMany, B = index_bits<K, E>();
  if ((int)blockIdx.x >= tiles) {
    fill_part(fill, blockIdx.x - tiles);
    return;
  }
  __shared__ K lds[2 * kTile];
  const int64_t base = (int64_t)blockIdx.x * kTile;
  const int count = n - base < kTile ? (int)(n - base) : kTile;
  K v[E];
  load_tile<K, E>(token + base, count, rows, v);
  block_sort<K, E>(v, lds, kTile);
  const int first = threadIdx.x * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (first + e < count) {
      key[base + first + e] = (int32_t)(v[e] >> B);
      pos[base + first + e] =
          (int32_t)(base + ((uint32_t)v[e] & (uint32_t)(((uint64_t)1 << B) - 1)));
    }
  }
}

struct MergeParams {
  int64_t n, run;  // tokens, length of a sorted run (the last may be shorter)
  int fan;         // runs that make one
  const int32_t *key_in, *pos_in;
  int32_t *key_out, *pos_out;
  int blocks;      // merging workgroups; further ones fill
};

// A workgroup places 64 neighbouring tokens of one run at a time: each of its
// waves searches for them in every kMergeWaves-th run, kSearches runs at a time,
// so that few steps wait for one another, and the waves' counts are added.
__global__ __launch_bounds__(kMergeThreads) void merge_kernel(MergeParams p, Fill fill) {
  if ((int)blockIdx.x >= p.blocks) {
    fill_part(fill, (int)blockIdx.x - p.blocks);
    return;
  }
  __shared__ int32_t counts[kMergeWaves][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t run = p.run, span = run * p.fan;
  uint32_t top = 1;
  while ((int64_t)top * 2 <= run) top *= 2;
  // (a run is a multiple of 64)
  for (int64_t i0 = (int64_t)blockIdx.x * kWave; i0 < p.n; i0 += (int64_t)p.blocks * kWave) {
    const bool there = i0 + lane < p.n;
    const int64_t base = i0 / span * span;
    const int mine = (int)((i0 - base) / run);
    const int32_t key = there ? p.key_in[i0 + lane] : 0;
    const int64_t left = (p.n - base + run - 1) / run;
    const int fan = left < p.fan ? (int)left : p.fan;
    uint32_t before = 0;
    for (int q0 = wave; q0 < fan; q0 += kSearches * kMergeWaves) {
      // tokens of run q that come before this one: those of lower rows, and in
      // the runs before its own those of its row too
      const char *a[kSearches];
      uint32_t len[kSearches], at[kSearches];
      int32_t limit[kSearches];
#pragma unroll
      for (int u = 0; u < kSearches; ++u) {
        const int q = q0 + u * kMergeWaves;
        const bool search = q < fan && q != mine;
        const int64_t start = base + (search ? q : 0) * run;
        a[u] = (const char *)(p.key_in + start);
        len[u] = search ? (uint32_t)(p.n - start < run ? p.n - start : run) : 0;
        limit[u] = key + (q < mine ? 1 : 0);
        at[u] = 0;
      }
      for (uint32_t s = top; s > 0; s >>= 1) {
        int32_t got[kSearches];
#pragma unroll
        for (int u = 0; u < kSearches; ++u)
          if (len[u] > 0)  // (index 0: in range, not used)
            got[u] = *(const int32_t *)(a[u] + (at[u] + s <= len[u] ? at[u] + s - 1 : 0u) * 4u);
#pragma unroll
        for (int u = 0; u < kSearches; ++u)
          if (len[u] > 0) at[u] += at[u] + s <= len[u] && got[u] < limit[u] ? s : 0;
      }
#pragma unroll
      for (int u = 0; u < kSearches; ++u) before += at[u];
    }
    counts[wave][lane] = (int32_t)before;
    __syncthreads();
    if (wave == 0 && there) {
      int64_t to = i0 + lane - mine * run;  // base and the place in its own run
#pragma unroll
      for (int w = 0; w < kMergeWaves; ++w) to += counts[w][lane];
      p.key_out[to] = key;
      p.pos_out[to] = p.pos_in[i0 + lane];
    }
    __syncthreads();  // counts are read before the next tokens' are written
  }
}

struct ReduceParams {
  GradParams g;
  const int32_t *key, *pos;  // sorted
  float *head, *tail;        // partial sums, one row of dim each per part
  int64_t parts;
  int part;                  // tokens per part: rounds of lane groups * per
  int log2g;                 // lanes per group
  int slices;                // column slices of 8 << log2g
};

template <typename TG, typename TO, int PER>
__global__ __launch_bounds__(kReduceThreads) void reduce_kernel(ReduceParams p) {
  __shared__ uint32_t keys[kMaxPart + 2];  // from the token before the part on
  __shared__ uint32_t where[kMaxPart];
  __shared__ f32x4_t heads[2 * kReduceThreads];
  __shared__ f32x4_t carry[2][2][kWave];   // the open row's sum, by round parity
  const GradParams &g = p.g;
  for (int64_t item = blockIdx.x; item < p.parts * p.slices; item += gridDim.x) {
    const int64_t part = item / p.slices, s0 = part * p.part;
    const Lanes l = lanes_of(p.log2g, item - part * p.slices, g.dim);
    const int lane = threadIdx.x & ((1 << p.log2g) - 1);
    int nv = 0;  // tokens of the part that are in the table
    for (int i = threadIdx.x; i < p.part + 2; i += kReduceThreads) {
      const int64_t s = s0 + i - 1;
      keys[i] = s >= 0 && s < g.n ? (uint32_t)p.key[s] : (uint32_t)g.rows;
      if (i < p.part && s + 1 < g.n) where[i] = (uint32_t)p.pos[s + 1];
    }
    __syncthreads();
    for (int i = threadIdx.x; i - (int)threadIdx.x < p.part; i += kReduceThreads)
      nv += __syncthreads_count(i < p.part && keys[1 + (i < p.part ? i : 0)] < (uint32_t)g.rows);
    auto key = [&](int i) { return keys[1 + i]; };
    // a row that began in an earlier part (no token has the row number rows)
    const uint32_t earlier = nv > 0 && s0 > 0 && keys[0] == keys[1] ? keys[0] : (uint32_t)g.rows;
    const bool leaves = nv == p.part && keys[nv + 1] == keys[nv];
    int round = 0;
    for (int t0 = 0; t0 < nv; t0 += l.groups * PER, round ^= 1) {
      const int t1 = t0 + l.groups * PER < nv ? t0 + l.groups * PER : nv;
      const bool last = t1 == nv;
      reduce_tokens<TG, PER>(
          g, l, t0, t1, t0 > 0 ? key(t0 - 1) == key(t0) : earlier == key(0),
          last ? leaves : key(t1 - 1) == key(t1), heads, key, [&](int i) { return where[i]; },
          [&](float (&acc)[8]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[e] = t0 > 0 ? carry[round][0][lane][e] : 0.0f;
              acc[4 + e] = t0 > 0 ? carry[round][1][lane][e] : 0.0f;
            }
          },
          [&](uint32_t row, const float (&acc)[8]) {
            if (last) {
              store_chunk<F32>((row == earlier ? p.head : p.tail) + part * g.dim, l.c, g.dim, acc);
            } else {
              carry[round ^ 1][0][lane] = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
              carry[round ^ 1][1][lane] = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
            }
          },
          [&](uint32_t row, const float (&acc)[8]) {
            if (row == earlier)
              store_chunk<F32>(p.head + part * g.dim, l.c, g.dim, acc);
            else
              finish_row<TO>(g, row, l.c, acc);
          });
      __syncthreads();  // heads are read before the next round writes them
    }
    __syncthreads();  // before the next item's keys
  }
}

// Adds the partial sums of a row that crosses parts: the workgroup of the part
// in which the row begins (the others end at once).  Partial 0 is that part's
// tail, partial k the head of the k-th part after it.  Each lane group adds a
// run of them, and the groups' sums are joined in order through LDS.
template <typename TO>
__global__ __launch_bounds__(kFixThreads) void fix_kernel(ReduceParams p) {
  const GradParams &g = p.g;
  const int G = 1 << p.log2g;
  const Lanes l = lanes_of(p.log2g, blockIdx.y, g.dim);
  __shared__ f32x4_t sums[2][kFixThreads];
  for (int64_t part = blockIdx.x; part < p.parts; part += gridDim.x) {
    const int64_t s0 = part * p.part, s1 = s0 + p.part;
    if (s1 >= g.n) return;  // the last part
    const int32_t row = p.key[s1 - 1];
    const int32_t next = p.key[s1], first = p.key[s0], before = s0 > 0 ? p.key[s0 - 1] : -1;
    if (row >= g.rows || next != row || (first == row && before == row)) continue;
    int64_t n = 0;  // parts after this one that the row reaches
    for (;;) {
      const int64_t s = s1 + (n + threadIdx.x) * p.part;
      const int got = __syncthreads_count(s < g.n && p.key[s] == row);
      n += got;
      if (got < kFixThreads) break;
    }
    const int64_t each = (n + 1 + l.groups - 1) / l.groups;
    const int64_t k0 = l.group * each, k1 = k0 + each < n + 1 ? k0 + each : n + 1;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    if (l.live) {
      for (int64_t k = k0; k < k1; k += kUnroll) {
        float v[kUnroll][8];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
          if (k + j < k1)
            load_chunk<F32>((k + j == 0 ? p.tail : p.head) + (part + k + j) * g.dim, l.c, g.dim,
                            v[j]);
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
          if (k + j < k1)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += v[j][e];
      }
    }
    // the groups' sums, neighbours first
    for (int half = 1; half < l.groups && half <= n; half *= 2) {
      sums[0][threadIdx.x] = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
      sums[1][threadIdx.x] = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
      __syncthreads();
      if (l.group % (2 * half) == 0) {
        const f32x4_t lo = sums[0][threadIdx.x + half * G], hi = sums[1][threadIdx.x + half * G];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[e] += lo[e];
          acc[4 + e] += hi[e];
        }
      }
      __syncthreads();
    }
    if (l.group == 0 && l.live) finish_row<TO>(g, (uint32_t)row, l.c, acc);
  }
}

// ---------------------------------------------------------------- launch --

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// log2 of the lanes that hold a row: 8 elements each, up to `most`.
int lane_group_log2(int dim, int most) {
  int g = 0;
  while ((8 << g) < dim && g < most) ++g;
  return g;
}

struct Layout {
  int levels, fan;
  int log2g, slices, per, part;
  int64_t parts;
  int64_t key[2], pos[2], head, tail, total;  // byte offsets
};

Layout plan_layout(int64_t n, int64_t rows, int dim) {
  (void)rows;
  Layout l{};
  const int64_t tiles = (n + kTile - 1) / kTile;
  l.levels = tiles <= kOneMerge ? 1 : 0;
  if (tiles > kOneMerge)
    for (int64_t all = 1; all < tiles; all *= kMaxFan) ++l.levels;
  l.fan = 1;
  for (;; ++l.fan) {  // the least fan whose power reaches all tiles
    int64_t all = 1;
    for (int i = 0; i < l.levels; ++i) all *= l.fan;
    if (all >= tiles) break;
  }
  l.log2g = lane_group_log2(dim, 6);
  l.slices = (dim + (8 << l.log2g) - 1) / (8 << l.log2g);
  const int groups = kReduceThreads >> l.log2g;
  l.per = kMaxPer;
  while (l.per > 2 && n / ((int64_t)groups * l.per) * l.slices < 1024) l.per /= 2;
  // long parts leave fewer partial sums: as long as 1024 workgroups remain
  l.part = groups * l.per;
  while (l.part * 2 <= kMaxPart && n / (l.part * 2) * l.slices >= 1024) l.part *= 2;
  l.parts = (n + l.part - 1) / l.part;
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
  l.head = take(l.parts * dim * 4);
  l.tail = take(l.parts * dim * 4);
  l.total = at;
  return l;
}

Fill part_of(const GradParams &g, int out_bytes, int part, int parts, int threads) {
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
    const int64_t want = (f.width * out_bytes / 16 + threads - 1) / threads;
    const int64_t most = (int64_t)kFillBlocks * kThreads / threads;
    f.blocks = (int)(want < 1 ? 1 : want < most ? want : most);
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

template <typename TG, typename TO, typename K, int E>
void launch_small(const GradParams &g, hipStream_t stream) {
  SmallParams p{};
  p.g = g;
  p.P = kWave * E;
  while (p.P < g.n) p.P *= 2;
  // 64 columns to a workgroup, and as many parts of the tokens as make 1024
  // workgroups: all sort the same tokens, so more would only sort more often
  p.log2g = lane_group_log2(g.dim, 3);
  while (p.log2g < 6 && (g.dim + (8 << p.log2g) - 1) / (8 << p.log2g) > 64) ++p.log2g;
  p.slices = (g.dim + (8 << p.log2g) - 1) / (8 << p.log2g);
  const int groups = kThreads >> p.log2g;
  const int64_t most = (g.n + groups - 1) / groups, fit = 1024 / p.slices;
  p.segments = (int)(most < 1 ? 1 : fit < 1 ? 1 : most < fit ? most : fit);
  int64_t blocks = (int64_t)p.segments * p.slices;
  if (!g.accumulate) {  // further ones for the rows that no token names
    int64_t fill = g.rows * g.dim * (int64_t)sizeof(typename TO::S) / (kThreads * 64);
    if (fill > kFillBlocks) fill = kFillBlocks;
    if (fill > g.rows) fill = g.rows;
    blocks += fill < 1 ? 1 : fill;
  }
  launch_kernel(small_kernel<TG, TO, K, E>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
}

template <typename TG, typename TO>
hipError_t launch_typed(const GradParams &g, void *ws, hipStream_t stream) {
  if (g.n <= kTile) {
    if (g.n <= kFew * kThreads) {
      if (g.rows < kRows32<kFew>)
        launch_small<TG, TO, uint32_t, kFew>(g, stream);
      else
        launch_small<TG, TO, uint64_t, kFew>(g, stream);
    } else if (g.rows < kRows32<kMany>) {
      launch_small<TG, TO, uint32_t, kMany>(g, stream);
    } else {
      launch_small<TG, TO, uint64_t, kMany>(g, stream);
    }
    return hipGetLastError();
  }
  const int ob = (int)sizeof(typename TO::S);
  uint8_t *w = (uint8_t *)ws;
  const Layout l = plan_layout(g.n, g.rows, g.dim);
  const int fills = 1 + l.levels;
  int32_t *key = (int32_t *)(w + l.key[0]), *pos = (int32_t *)(w + l.pos[0]);
  const int tiles = (int)((g.n + kTile - 1) / kTile);
  Fill f = part_of(g, ob, 0, fills, kThreads);
  const dim3 grid((unsigned)(tiles + f.blocks)), block(kThreads);
  // each launch reads what the one before wrote: none follows one that failed
  hipError_t err;
  if (g.rows < kRows32<kMany>)
    launch_kernel(tile_sort_kernel<uint32_t>, grid, block, 0, stream, g.token, g.n, g.rows, tiles,
                  key, pos, f);
  else
    launch_kernel(tile_sort_kernel<uint64_t>, grid, block, 0, stream, g.token, g.n, g.rows, tiles,
                  key, pos, f);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  MergeParams m{};
  m.n = g.n;
  m.run = kTile;
  m.fan = l.fan;
  const int64_t groups = (g.n + kWave - 1) / kWave;
  m.blocks = (int)(groups < kMergeBlocks ? groups : kMergeBlocks);
  for (int level = 0; level < l.levels; ++level) {
    m.key_in = (const int32_t *)(w + l.key[level & 1]);
    m.pos_in = (const int32_t *)(w + l.pos[level & 1]);
    m.key_out = (int32_t *)(w + l.key[(level + 1) & 1]);
    m.pos_out = (int32_t *)(w + l.pos[(level + 1) & 1]);
    f = part_of(g, ob, 1 + level, fills, kMergeThreads);
    launch_kernel(merge_kernel, dim3((unsigned)(m.blocks + f.blocks)), dim3(kMergeThreads), 0,
                  stream, m, f);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    m.run *= l.fan;
  }
  ReduceParams rp{};
  rp.g = g;
  rp.key = (const int32_t *)(w + l.key[l.levels & 1]);
  rp.pos = (const int32_t *)(w + l.pos[l.levels & 1]);
  rp.head = (float *)(w + l.head);
  rp.tail = (float *)(w + l.tail);
  rp.parts = l.parts;
  rp.part = l.part;
  rp.log2g = l.log2g;
  rp.slices = l.slices;
  const int64_t items = l.parts * l.slices;
  const dim3 reduce_grid((unsigned)(items < kMaxBlocks ? items : kMaxBlocks));
  if (l.per == 8)
    launch_kernel(reduce_kernel<TG, TO, 8>, reduce_grid, dim3(kReduceThreads), 0, stream, rp);
  else if (l.per == 4)
    launch_kernel(reduce_kernel<TG, TO, 4>, reduce_grid, dim3(kReduceThreads), 0, stream, rp);
  else
    launch_kernel(reduce_kernel<TG, TO, 2>, reduce_grid, dim3(kReduceThreads), 0, stream, rp);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  const int64_t blocks = l.parts * l.slices < kMaxBlocks ? l.parts : kMaxBlocks / l.slices;
  launch_kernel(fix_kernel<TO>, dim3((unsigned)blocks, l.slices), dim3(kFixThreads), 0, stream, rp);
  return hipGetLastError();
}

}  // namespace

size_t lookup_grad_workspace(int64_t n, int64_t rows, int dim) {
  return n > kTile ? (size_t)plan_layout(n, rows, dim).total : 0;
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
