// Embedding lookup and its gradient.
//
//   out[i] = scale * table[tokens[i]]
//   dW[v]  = scale * tree(grad[p] : tokens[p] == v, p ascending)
//
// The gradient is a reduction per token, and takes the library's expression
// for one: the shift-reduce tree over the rows in order. Equal tokens are
// brought together by a stable counting sort (integers only, so its result is
// unique), then every row of the table is one tree.
//
// Measured, bf16: lookup of 32,805 rows of 4096 columns in a table of 65,536,
// 68 us (537 MB at 7.9 TB/s, since repeated rows come from L2); gradient of
// 65,536 rows of 2048 columns into 65,536 rows, the most frequent token 4,096
// times, 210 us against 119 us for its 806 MB at the copy rate (its launches
// one by one, with the events around them: 23 us sort, 153 us rows and parts,
// 39 us long rows).
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

// ------------------------------------------------------------- lookup
// Bound by DRAM; few tokens are bound by the call (4 us).
// A block covers blockDim.y tokens; the threads of a row walk its columns, V at
// a time: neighbours in one access (kWide), or blockDim.x apart, so that the
// threads' accesses are consecutive.
template <class T, int V, bool kWide>
__global__ void __launch_bounds__(256)
embedding_kernel(const void* __restrict__ tokens, int index_bytes, int64_t n,
                 const T* __restrict__ table, int64_t vocab, int64_t dim, int64_t row_stride,
                 float scale, T* __restrict__ out, int64_t out_stride) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (i >= n) return;
  const int64_t v = load_index(tokens, index_bytes, i);
  const bool real = v >= 0 && v < vocab;
  const T* src = table + (real ? v : 0) * row_stride;
  T* dst = out + i * out_stride;
  const int tx = threadIdx.x, nx = blockDim.x;
  if (kWide) {
    for (int64_t c = (int64_t)tx * V; c < dim; c += (int64_t)nx * V) {
      const int have = (int)min((int64_t)V, dim - c);
      float f[V];
      if (real) {
        load_f32<T, V>(src + c, have == V, have, f);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = f[k] * scale;
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = 0.0f;
      }
      store_f32<T, V>(dst + c, have == V, have, f);
    }
  } else {
    for (int64_t c = tx; c < dim; c += (int64_t)nx * V) {
      float f[V];
#pragma unroll
      for (int k = 0; k < V; ++k)
        f[k] = real && c + k * nx < dim ? to_f32(src[c + k * nx]) * scale : 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (c + k * nx < dim) dst[c + k * nx] = from_f32<T>(f[k]);
    }
  }
}

// --------------------------------------------------------------- sort
constexpr int kSortThreads = 1024;  // most
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRows = 1024;  // most rows a block sorts: 128 KB of counters
constexpr int kSortBatch = 8;    // tokens a lane has in flight
constexpr int kSortKept = 256;   // a warp's tokens that need no second look
constexpr int kLong = 16;        // positions of a long row, and of a part of its tree

// Where the sort puts things.
struct Sorted {
  int32_t* row_start;  // [vocab + 1]
  int32_t* order;      // [n]: positions by (token, position)
  int32_t* part;       // [n / kLong]: where a part of a long row begins, or -1
  int32_t* part_row;   // [n / kLong]: the row whose first part this is, or -1
};

// Tokens at p, p + 32, ...; -1 for those outside [0, vocab).
__device__ __forceinline__ void load_tokens(const void* tokens, int index_bytes, int64_t p,
                                            int64_t end, int64_t vocab, int32_t (&v)[kSortBatch]) {
  if (index_bytes == 8) {
    int64_t q[kSortBatch];
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j)
      q[j] = p + j * 32 < end ? static_cast<const int64_t*>(tokens)[p + j * 32] : -1;
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j) v[j] = q[j] >= 0 && q[j] < vocab ? (int32_t)q[j] : -1;
  } else {
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j)
      v[j] = p + j * 32 < end ? static_cast<const int32_t*>(tokens)[p + j * 32] : -1;
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j) v[j] = v[j] >= 0 && v[j] < vocab ? v[j] : -1;
  }
}

// Stable counting sort of the positions by token. Block j owns the rows
// [j R, (j+1) R) and reads every token, so that it needs nothing of another
// block: the number of smaller tokens is where its part of `order` begins.
// Warp w owns the w-th contiguous part of the positions in both sweeps; its
// counters are its own, and within 32 positions equal tokens are ranked by
// lane, so the order is that of the positions. All counts are integers: the
// result is unique whatever the order of the atomics. Every block reading all
// tokens costs L2 reads (65,536 tokens: 152 x 512 KB a sweep, of a sort of
// 23 us in all) and saves the launches and the traffic of a sort by digits; a
// warp's own tokens are kept from the first sweep, which spares most warps the
// second.
//
// A row with kLong positions or more has its complete groups of kLong summed
// by blocks of their own. Group k of the row that begins at s is number
// s / kLong + k: two rows' numbers never meet, and a block's rows have theirs
// between its ends' quotients.
__global__ void __launch_bounds__(kSortThreads)
token_sort_kernel(const void* __restrict__ tokens, int index_bytes, int64_t n, int64_t vocab,
                  int rows_per_block, Sorted out) {
  extern __shared__ int32_t count[];  // [warp][row], then cursors
  __shared__ uint32_t kept_s[kSortWarps][kSortKept];  // (offset in the warp's share, row)
  __shared__ int32_t warp_total[kSortWarps];
  __shared__ int32_t base_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads / 32;  // at least R threads
  const int32_t lo = (int32_t)((int64_t)blockIdx.x * rows_per_block);
  const int32_t hi = (int32_t)min(vocab, (int64_t)lo + rows_per_block);
  const int R = hi - lo;
  for (int k = tid; k < R * warps; k += threads) count[k] = 0;
  if (tid == 0) base_s = 0;
  __syncthreads();

  constexpr int kStep = 32 * kSortBatch;
  const int64_t share = (n + warps - 1) / warps + 31;
  const int64_t p0 = min(n, warp * (share / 32 * 32)), p1 = min(n, p0 + share / 32 * 32);
  int32_t* mine = count + warp * R;
  uint32_t* kept = kept_s[warp];
  int32_t below = 0, hits = 0;
  for (int64_t p = p0 + lane; p - lane < p1; p += kStep) {
    int32_t v[kSortBatch];
    load_tokens(tokens, index_bytes, p, p1, vocab, v);
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j) {
      if (v[j] >= 0 && v[j] < lo) ++below;
      const bool in = v[j] >= lo && v[j] < hi;
      const uint32_t any = __ballot_sync(~0u, in);
      if (in) {
        const int at = hits + __popc(any & ((1u << lane) - 1));
        if (at < kSortKept) kept[at] = (uint32_t)(p + j * 32 - p0) << 10 | (uint32_t)(v[j] - lo);
        atomicAdd(&mine[v[j] - lo], 1);
      }
      hits += __popc(any);
    }
  }
  below = __reduce_add_sync(~0u, below);
  if (lane == 0) atomicAdd(&base_s, below);
  __syncthreads();
  const int32_t base = base_s;

  // Exclusive prefix over the rows of their totals, and within a row over the
  // warps: thread r takes row r.
  int32_t total = 0;
  if (tid < R)
    for (int w = 0; w < warps; ++w) total += count[w * R + tid];
  int32_t incl = total;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const int32_t o = __shfl_up_sync(~0u, incl, s);
    if (lane >= s) incl += o;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  int32_t before = base, all = base;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += warp_total[w];
    all += warp_total[w];
  }
  const int32_t start = before + incl - total;
  if (tid < R) {
    out.row_start[lo + tid] = start;
    if (lo + tid == vocab - 1) out.row_start[vocab] = start + total;
    int32_t at = start;
    for (int w = 0; w < warps; ++w) {
      const int32_t c = count[w * R + tid];
      count[w * R + tid] = at;
      at += c;
    }
  }
  const int32_t parts_end = hi == vocab ? (int32_t)(n / kLong) : all / kLong;
  for (int32_t k = base / kLong + tid; k < parts_end; k += threads)
    out.part[k] = out.part_row[k] = -1;
  __syncthreads();
  for (int32_t k = 0; k < total / kLong; ++k) out.part[start / kLong + k] = start + k * kLong;
  if (total >= kLong) out.part_row[start / kLong] = lo + tid;

  // places 32 positions, those lanes' with `in`, in lane order
  auto place = [&](bool in, int r, int32_t p) {
    const uint32_t any = __ballot_sync(~0u, in);
    if (any == 0) return;
    if (in) {
      const uint32_t same = __match_any_sync(any, r);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int32_t at = mine[r];
      __syncwarp(any);
      if (rank == 0) mine[r] = at + __popc(same);
      out.order[at + rank] = p;
    }
    __syncwarp();
  };
  if (hits <= kSortKept && share < (1 << 22)) {
    for (int k = 0; k < hits; k += 32) {
      const uint32_t q = k + lane < hits ? kept[k + lane] : 0;
      place(k + lane < hits, q & 1023u, (int32_t)(p0 + (q >> 10)));
    }
  } else {
    for (int64_t p = p0 + lane; p - lane < p1; p += kStep) {
      int32_t v[kSortBatch];
      load_tokens(tokens, index_bytes, p, p1, vocab, v);
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j)
        place(v[j] >= lo && v[j] < hi, v[j] - lo, (int32_t)(p + j * 32));
    }
  }
}

// ---------------------------------------------------------- row trees
constexpr int kRowGroup = 8;    // gradient rows read at a time
constexpr int kRowLevels = 28;  // of the tree above a group of parts

template <class T>
struct Grad {
  const T* p;
  int64_t stride;
};

// A lane's four columns among 128 of a warp: neighbours, read and written at
// once (kWide: rows of the gradient and of the table allow it), or 32 apart,
// so that the warp's accesses are consecutive. Columns are summed by
// themselves, so this changes no result.
template <bool kWide>
struct Columns {
  static constexpr int kStep = kWide ? 1 : 32;
  static __device__ __forceinline__ int first(int lane) { return kWide ? lane * 4 : lane; }
  static __device__ __forceinline__ int have(int64_t c, int64_t dim) {
    return (int)max((int64_t)0, min((int64_t)4, (dim - c + kStep - 1) / kStep));
  }
};
template <class T, bool kWide>
using Four = Raw<T, 4, kWide, Columns<kWide>::kStep, !kWide>;

template <class T, bool kWide>
__device__ __forceinline__ void read_four(const T* p, int have, float (&f)[4]) {
  Four<T, kWide> r;
  r.load(p, have == 4, have);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = r.get(j);
}
template <bool kWide>
__device__ __forceinline__ void write_four(float* p, int have, const float (&f)[4]) {
  store_raw<float, 4, kWide, Columns<kWide>::kStep>(p, have == 4, have, f);
}

// The perfect tree over kRowGroup values a column.
__device__ __forceinline__ void group_tree(float (&g)[kRowGroup][4]) {
#pragma unroll
  for (int s = 1; s < kRowGroup; s *= 2)
#pragma unroll
    for (int k = 0; k < kRowGroup; k += 2 * s)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[k][j] = add_rn(g[k][j], g[k + s][j]);
}

// The parts of long rows: a warp takes one and 512 columns, 128 at a time.
constexpr int kPartSteps = 4, kPartColumns = 128 * kPartSteps;
template <class T, bool kWide>
__device__ __forceinline__ void sum_part(const Grad<T>& grad, const Sorted& in, int64_t item,
                                         int64_t dim, int64_t part_warps, float* sums) {
  const int lane = threadIdx.x % 32;
  int64_t c0;
  const int64_t k = divide(item, part_warps, c0);
  const int32_t first = in.part[k];
  if (first < 0) return;
  c0 = c0 * kPartColumns + Columns<kWide>::first(lane);
  const int32_t at = in.order[first + lane % kLong];
  const int64_t pitch = (dim + 3) / 4 * 4;
#pragma unroll 1
  for (int i = 0; i < kPartSteps; ++i) {
    const int64_t c = c0 + i * 128;
    const int have = Columns<kWide>::have(c, dim);
    Four<T, kWide> raw[kLong];
#pragma unroll
    for (int q = 0; q < kLong; ++q)
      raw[q].load(grad.p + __shfl_sync(~0u, at, q) * grad.stride + c, have == 4, have);
    float g[2][kRowGroup][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int q = 0; q < kRowGroup; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) g[h][q][j] = raw[h * kRowGroup + q].get(j);
      group_tree(g[h]);
    }
    static_assert(kLong == 2 * kRowGroup, "a part is two groups");
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = add_rn(g[0][0][j], g[1][0][j]);
    write_four<kWide>(sums + k * pitch + c, have, f);
  }
}

// The tree over the first t (1 to 7) of the values a column, in v.
__device__ __forceinline__ void tail_tree(const float (&g)[kRowGroup][4], int t, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a01 = add_rn(g[0][j], g[1][j]), a45 = add_rn(g[4][j], g[5][j]);
    const float a03 = add_rn(a01, add_rn(g[2][j], g[3][j]));
    const float left = t >= 4 ? a03 : t >= 2 ? a01 : g[0][j];
    const float right = t == 3 ? g[2][j] : t == 5 ? g[4][j] : t == 6 ? a45 : add_rn(a45, g[6][j]);
    v[j] = (t == 3 || t >= 5) ? add_rn(left, right) : left;
  }
}

struct Table {
  float* dw;
  int64_t stride;
  float scale;
  bool accumulate;

  template <bool kWide>
  __device__ __forceinline__ void put(int64_t v, int64_t c, int have, float (&acc)[4]) const {
    float* dst = dw + v * stride + c;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = acc[j] * scale;
    if (accumulate) {
      float old[4];
      read_own<float, 4, kWide, Columns<kWide>::kStep>(dst, have == 4, have, old);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = add_rn(old[j], acc[j]);
    }
    write_four<kWide>(dst, have, acc);
  }
};

// A long row, 128 columns, by a warp: the parts' sums eight at a time with the
// next eight in flight, then the rows after them.
template <class T, bool kWide>
__device__ __forceinline__ void long_row(const Grad<T>& grad, const Sorted& in, const float* sums,
                                         int64_t begin, int32_t v, int64_t c, int64_t dim,
                                         const Table& out) {
  const int lane = threadIdx.x % 32;
  const int have = Columns<kWide>::have(c, dim);
  const int32_t first = in.row_start[v], count = in.row_start[v + 1] - first;
  const int32_t n = count / kLong, tail0 = first + n * kLong;
  const int rest = count % kLong, group = rest / kRowGroup, tail = rest % kRowGroup;
  const int32_t at = rest > 0 ? in.order[tail0 + min(lane, rest - 1)] : 0;
  const int64_t pitch = (dim + 3) / 4 * 4;
  const float* s = sums + begin * pitch + c;
  // the rows after the parts: a group of 8, and fewer than 8
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  Four<T, kWide> r[2][kRowGroup];
#pragma unroll
  for (int k = 0; k < kRowGroup; ++k) {
    const int64_t p = __shfl_sync(~0u, at, k) * grad.stride;
    const int64_t q = __shfl_sync(~0u, at, group * kRowGroup + k) * grad.stride;
    if (group > 0) r[0][k].load(grad.p + p + c, have == 4, have);
    if (k < tail) r[1][k].load(grad.p + q + c, have == 4, have);
  }
  bool has = tail > 0;
  if (has) {
    float g[kRowGroup][4];
#pragma unroll
    for (int k = 0; k < kRowGroup; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[k][j] = r[1][k].get(j);
    tail_tree(g, tail, acc);
  }
  if (group > 0) {
    float g[kRowGroup][4];
#pragma unroll
    for (int k = 0; k < kRowGroup; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[k][j] = r[0][k].get(j);
    group_tree(g);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = has ? add_rn(g[0][j], acc[j]) : g[0][j];
    has = true;
  }
  // the parts: complete groups of 8 onto a stack (in local memory, an access a
  // group), the others folded first
  float stack[kRowLevels][4];
  const int32_t groups = n / kRowGroup;
  float next[kRowGroup][4];  // of the group after this one
  auto load = [&](int32_t i) {
    const int many = i < groups ? kRowGroup : n % kRowGroup;
#pragma unroll
    for (int k = 0; k < kRowGroup; ++k)
      if (k < many) read_four<float, kWide>(s + (i * kRowGroup + k) * pitch, have, next[k]);
  };
  load(0);
#pragma unroll 1
  for (int32_t i = 0; i <= groups; ++i) {
    const int many = i < groups ? kRowGroup : n % kRowGroup;
    float g[kRowGroup][4];
#pragma unroll
    for (int k = 0; k < kRowGroup; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[k][j] = next[k][j];
    if (i < groups) load(i + 1);
    if (i < groups) {
      group_tree(g);
      int lv = 0;
      for (; (i >> lv) & 1; ++lv)
#pragma unroll
        for (int j = 0; j < 4; ++j) g[0][j] = add_rn(stack[lv][j], g[0][j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) stack[lv][j] = g[0][j];
    } else if (many > 0) {
      // shift-reduce of fewer than 8, folded onto what lies to the right
      float a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a01 = add_rn(g[0][j], g[1][j]), a23 = add_rn(g[2][j], g[3][j]);
        const float a45 = add_rn(g[4][j], g[5][j]);
        a[j] = acc[j];
        bool h = has;
        if (many & 1) {
          const float one = many == 1 ? g[0][j] : many == 3 ? g[2][j] : many == 5 ? g[4][j] : g[6][j];
          a[j] = h ? add_rn(one, a[j]) : one;
          h = true;
        }
        if (many & 2) {
          const float two = many >= 6 ? a45 : a01;
          a[j] = h ? add_rn(two, a[j]) : two;
          h = true;
        }
        if (many & 4) {
          const float four = add_rn(a01, a23);
          a[j] = h ? add_rn(four, a[j]) : four;
        }
        acc[j] = a[j];
      }
      has = true;
    }
  }
  for (int lv = 0; (groups >> lv) != 0; ++lv) {
    if ((groups >> lv) & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = has ? add_rn(stack[lv][j], acc[j]) : stack[lv][j];
      has = true;
    }
  }
  if (have > 0) out.template put<kWide>(v, c, have, acc);
}

// The long rows: a warp takes 128 columns of those that begin among kLongParts
// parts (4,096 parts of 2048 columns, 370 rows, the longest of 4,096
// positions: 40 us with 8 parts or one a warp; 123 us with 32 parts a block,
// where rows wait for one another).
constexpr int kLongParts = 8;
template <class T, bool kWide>
__global__ void __launch_bounds__(256)
embedding_long_kernel(Grad<T> grad, Sorted in, const float* __restrict__ sums, int64_t parts,
                      int64_t dim, int64_t long_warps, Table out) {
  const int lane = threadIdx.x % 32;
  const int64_t item = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  int64_t c;
  const int64_t k = divide(item, long_warps, c) * kLongParts;
  c = c * 128 + Columns<kWide>::first(lane);
  const int32_t v = lane < kLongParts && k + lane < parts ? in.part_row[k + lane] : -1;
  for (uint32_t todo = __ballot_sync(~0u, v >= 0); todo != 0; todo &= todo - 1) {
    const int i = __ffs(todo) - 1;
    long_row<T, kWide>(grad, in, sums, k + i, __shfl_sync(~0u, v, i), c, dim, out);
  }
}

// The other rows: a warp takes one and kRowSteps times 128 columns, so that
// a row of one position, the most frequent length, has kRowSteps reads in
// flight behind the two that find it. Bound by DRAM and by those reads' latency
// (4 steps and 4 blocks an SM measured 127 us of rows alone where 2 steps took
// 155, 3 blocks 134). The first blocks take the parts of the
// long rows, which need no more than the sort either.
#ifndef CR_EMBEDDING_STEPS
#define CR_EMBEDDING_STEPS 4
#endif
#ifndef CR_EMBEDDING_BLOCKS
#define CR_EMBEDDING_BLOCKS 4
#endif
constexpr int kRowSteps = CR_EMBEDDING_STEPS, kRowColumns = 128 * kRowSteps;
template <class T, bool kWide>
__global__ void __launch_bounds__(256, CR_EMBEDDING_BLOCKS)
embedding_rows_kernel(Grad<T> grad, Sorted in, int64_t part_items, int64_t part_warps,
                      float* __restrict__ sums, int64_t vocab, int64_t dim, int64_t row_warps,
                      Table out) {
  const int lane = threadIdx.x % 32;
  int64_t item = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (item < part_items) {
    sum_part<T, kWide>(grad, in, item, dim, part_warps, sums);
    return;
  }
  item -= part_items;
  int64_t begin;  // of the warp's columns
  const int64_t v = divide(item, row_warps, begin);
  begin *= kRowColumns;
  const int64_t c0 = begin + Columns<kWide>::first(lane);
  if (v >= vocab) return;
  const int32_t first = in.row_start[v], count = in.row_start[v + 1] - first;
  if (count >= kLong || (count == 0 && out.accumulate)) return;
  const int steps = (int)min((int64_t)kRowSteps, (dim - begin + 127) / 128);
  const bool full = begin + steps * 128 <= dim;
  auto have = [&](int i) { return full ? 4 : Columns<kWide>::have(c0 + i * 128, dim); };
  float* dst = out.dw + v * out.stride + c0;
  if (count == 0) {
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      if (i < steps) {
        const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        write_four<kWide>(dst + i * 128, have(i), zero);
      }
    }
    return;
  }
  const int32_t at0 = in.order[first + min(lane, count - 1)];
  if (count == 1) {
    const T* src = grad.p + at0 * grad.stride + c0;
    Four<T, kWide> r[kRowSteps];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i)
      if (i < steps) r[i].load(src + i * 128, have(i) == 4, have(i));
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      if (i < steps) {
        float acc[4] = {r[i].get(0), r[i].get(1), r[i].get(2), r[i].get(3)};
        out.template put<kWide>(v, c0 + i * 128, have(i), acc);
      }
    }
    return;
  }
  const int groups = count / kRowGroup, tail = count % kRowGroup;  // at most one group
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    const T* src = grad.p + c0 + i * 128;
    const int hv = have(i);
    const bool w = hv == 4;
    float acc[4];
    if (tail > 0) {
      Four<T, kWide> r[kRowGroup];
#pragma unroll
      for (int k = 0; k < kRowGroup - 1; ++k) {
        const int32_t q = __shfl_sync(~0u, at0, groups * kRowGroup + k);
        if (k < tail) r[k].load(src + q * grad.stride, w, hv);
      }
      float g[kRowGroup][4];
#pragma unroll
      for (int k = 0; k < kRowGroup - 1; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) g[k][j] = r[k].get(j);
      tail_tree(g, tail, acc);
    }
    if (groups > 0) {
      Four<T, kWide> r[kRowGroup];
#pragma unroll
      for (int k = 0; k < kRowGroup; ++k)
        r[k].load(src + __shfl_sync(~0u, at0, k) * grad.stride, w, hv);
      float g[kRowGroup][4];
#pragma unroll
      for (int k = 0; k < kRowGroup; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) g[k][j] = r[k].get(j);
      group_tree(g);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = tail > 0 ? add_rn(g[0][j], acc[j]) : g[0][j];
    }
    out.template put<kWide>(v, c0 + i * 128, hv, acc);
  }
}

// ------------------------------------------------------- few positions
// Up to kFewTokens positions take one launch: a block sorts the positions of
// kFewRows rows of the table in shared memory and sums them, a warp a row and
// 128 columns at a time. A token's positions are summed by one warp for every
// 128 columns, one group of 8 after another, which the launches above share
// out: 2,048 equal tokens of 64 columns take 209 us here, where as many spread
// ones take 9 us and 2,049 equal ones, in three launches, 33 us. (The rule
// between the two knows sizes, not tokens.)
constexpr int kFewTokens = 2048, kFewRows = 16;
constexpr int kFewEach = kFewTokens / 256;  // tokens a thread

// One row, 128 columns: the tree over the `count` positions in `order`.
template <class T, bool kWide>
__device__ __forceinline__ void sum_row(const Grad<T>& grad, const int32_t* order, int count,
                                        int64_t c, int have, float (&acc)[4]) {
  const int groups = count / kRowGroup, tail = count % kRowGroup;
  bool has = tail > 0;
  if (has) {
    Four<T, kWide> r[kRowGroup];
#pragma unroll
    for (int k = 0; k < kRowGroup - 1; ++k)
      if (k < tail)
        r[k].load(grad.p + order[groups * kRowGroup + k] * grad.stride + c, have == 4, have);
    float g[kRowGroup][4];
#pragma unroll
    for (int k = 0; k < kRowGroup - 1; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[k][j] = r[k].get(j);
    tail_tree(g, tail, acc);
  }
  float stack[12][4];  // in local memory: an access a group of 8
#pragma unroll 1
  for (int i = 0; i < groups; ++i) {
    Four<T, kWide> r[kRowGroup];
#pragma unroll
    for (int k = 0; k < kRowGroup; ++k)
      r[k].load(grad.p + order[i * kRowGroup + k] * grad.stride + c, have == 4, have);
    float g[kRowGroup][4];
#pragma unroll
    for (int k = 0; k < kRowGroup; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[k][j] = r[k].get(j);
    group_tree(g);
    int lv = 0;
    for (; (i >> lv) & 1; ++lv)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[0][j] = add_rn(stack[lv][j], g[0][j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) stack[lv][j] = g[0][j];
  }
  for (int lv = 0; (groups >> lv) != 0; ++lv) {
    if ((groups >> lv) & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = has ? add_rn(stack[lv][j], acc[j]) : stack[lv][j];
      has = true;
    }
  }
}

template <class T, bool kWide>
__global__ void __launch_bounds__(256)
embedding_few_kernel(const void* __restrict__ tokens, int index_bytes, int n, Grad<T> grad,
                     int64_t vocab, int64_t dim, int col_warps, Table out) {
  __shared__ int32_t order[kFewTokens];
  __shared__ int32_t count[8][kFewRows];
  __shared__ int32_t starts[kFewRows + 1];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t lo = (int64_t)blockIdx.x * kFewRows;
  const int rows = (int)min((int64_t)kFewRows, vocab - lo);
  if (tid < 8 * kFewRows) count[tid / kFewRows][tid % kFewRows] = 0;
  // warp w takes the w-th share of the positions, as in the sort above
  const int share = ((n + 7) / 8 + 31) / 32 * 32, p0 = warp * share;
  int r[kFewEach];
#pragma unroll
  for (int j = 0; j < kFewEach; ++j) {
    const int q = j * 32 + lane, p = p0 + q;
    const int64_t v = q < share && p < n ? load_index(tokens, index_bytes, p) : -1;
    r[j] = v >= lo && v < lo + rows ? (int)(v - lo) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kFewEach; ++j)
    if (r[j] >= 0) atomicAdd(&count[warp][r[j]], 1);
  __syncthreads();
  if (warp == 0) {
    int total = 0;
    if (lane < kFewRows)
      for (int w = 0; w < 8; ++w) total += count[w][lane];
    int incl = total;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const int o = __shfl_up_sync(~0u, incl, s);
      if (lane >= s) incl += o;
    }
    if (lane < kFewRows) {
      int at = incl - total;
      starts[lane] = at;
      if (lane == kFewRows - 1) starts[kFewRows] = incl;
      for (int w = 0; w < 8; ++w) {
        const int c = count[w][lane];
        count[w][lane] = at;
        at += c;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kFewEach; ++j) {
    const bool in = r[j] >= 0;
    const uint32_t any = __ballot_sync(~0u, in);
    if (any == 0) continue;
    if (in) {
      const uint32_t same = __match_any_sync(any, r[j]);
      const int rank = __popc(same & ((1u << lane) - 1)), at = count[warp][r[j]];
      __syncwarp(any);
      if (rank == 0) count[warp][r[j]] = at + __popc(same);
      order[at + rank] = p0 + j * 32 + lane;
    }
    __syncwarp();
  }
  __syncthreads();

#pragma unroll 1
  for (int item = warp; item < rows * col_warps; item += 8) {
    const int row = item / col_warps;
    const int64_t c = (int64_t)(item - row * col_warps) * 128 + Columns<kWide>::first(lane);
    const int first = starts[row], many = starts[row + 1] - first;
    const int have = Columns<kWide>::have(c, dim);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (many > 0) {
      sum_row<T, kWide>(grad, order + first, many, c, have, acc);
      out.template put<kWide>(lo + row, c, have, acc);
    } else if (!out.accumulate) {
      write_four<kWide>(out.dw + (lo + row) * out.stride + c, have, acc);
    }
  }
}

int sort_rows(int64_t vocab) {
  int64_t r = ceil_div(vocab, 152);
  if (r < 1) r = 1;
  return (int)(r > kSortRows ? kSortRows : r);
}

}  // namespace
}  // namespace cr

extern "C" {

cr_status cr_embedding(const void* tokens, int32_t index_bytes, int64_t n, const void* table,
                       int64_t vocab, int64_t dim, int64_t row_stride, float scale, cr_dtype dt,
                       void* out, int64_t out_stride, void* stream) {
  using namespace cr;
  const size_t es = model_esize(dt);
  if (es == 0 || n < 0 || vocab < 0 || dim < 0 || !index_width_ok(index_bytes))
    return CR_ERR_INVALID_ARG;
  if (row_stride < dim || out_stride < dim) return CR_ERR_INVALID_ARG;
  if (n == 0 || dim == 0) return CR_OK;
  if (tokens == nullptr || out == nullptr || (vocab > 0 && table == nullptr) ||
      overwrites({out}, {tokens, table}))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(tokens, index_bytes) || !ptr_aligned(table, es) || !ptr_aligned(out, es))
    return CR_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = rows_aligned(table, row_stride, 0, es, 16) &&
                    rows_aligned(out, out_stride, 0, es, 16);
  const int v = (int)(16 / es);
  int tx = 1;
  while (tx < 256 && (int64_t)tx * v < dim) tx *= 2;
  const dim3 block(tx, 256 / tx);
  const int64_t blocks = ceil_div(n, block.y);
  if (blocks > kMaxBlocks) return CR_ERR_UNSUPPORTED;
  CR_MODEL_TYPE(dt, {
    constexpr int V = 16 / sizeof(T);
    CR_LAUNCH(kKEmbedding, s,
              (wide ? embedding_kernel<T, V, true> : embedding_kernel<T, V, false>)
              <<<(unsigned)blocks, block, 0, s>>>(
                  tokens, index_bytes, n, static_cast<const T*>(table), vocab, dim, row_stride,
                  scale, static_cast<T*>(out), out_stride));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

size_t cr_embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  using namespace cr;
  if (n < 0 || vocab < 0 || dim < 0 || n > INT32_MAX || vocab > INT32_MAX) return 0;
  return round256(((size_t)vocab + 1) * 4) + round256((size_t)n * 4) +
         2 * round256((size_t)(n / kLong) * 4) +
         round256((size_t)(n / kLong) * ((size_t)(dim + 3) / 4 * 4) * 4) + kStatusBytes;
}

cr_status cr_embedding_backward(const void* tokens, int32_t index_bytes, int64_t n,
                                const void* grad, int64_t grad_stride, int64_t vocab,
                                int64_t dim, float scale, cr_dtype dt, int32_t accumulate,
                                float* dw, int64_t dw_stride, void* ws, size_t ws_bytes,
                                void* stream) {
  using namespace cr;
  const size_t es = model_esize(dt);
  const size_t need = cr_embedding_backward_workspace_bytes(n, vocab, dim);
  if (es == 0 || need == 0 || !index_width_ok(index_bytes)) return CR_ERR_INVALID_ARG;
  if (grad_stride < dim || dw_stride < dim) return CR_ERR_INVALID_ARG;
  if (n > 0 && dim > 0 && (tokens == nullptr || grad == nullptr)) return CR_ERR_INVALID_ARG;
  if (vocab > 0 && dim > 0 && (dw == nullptr || overwrites({dw}, {tokens, grad})))
    return CR_ERR_INVALID_ARG;
  if ((tokens && !ptr_aligned(tokens, index_bytes)) || (grad && !ptr_aligned(grad, es)) ||
      (dw && !ptr_aligned(dw, 4)))
    return CR_ERR_INVALID_ARG;
  if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < need) return CR_ERR_WORKSPACE;
  if (vocab == 0 || dim == 0) return CR_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Table out = {dw, dw_stride, scale, accumulate != 0};
  const bool wide = rows_aligned(grad, grad_stride, 0, es, 4 * es) &&
                    rows_aligned(dw, dw_stride, 0, 4, 16);
  const int64_t row_warps = ceil_div(dim, kRowColumns), long_cols = ceil_div(dim, 128);
  // Few positions, thin on the table (at most 8192 elements of theirs a block
  // on average, since a block sums its rows alone): one launch instead of two
  // or three. Measured, one against three: 1,037 x 333 into 10,007 rows 14.3 and
  // 27.2 us; 600 x 256 into 5,000 8.5 and 23.4; 2,000 x 1024 into 60,000 58 and
  // 68; and beyond the rule 2,000 x 2000 into 3,000 57 and 29.
  const bool thin = n == 0 || dim <= (int64_t)512 * vocab / n;
  if (n <= kFewTokens && thin && long_cols <= INT32_MAX / kFewRows) {
    CR_MODEL_TYPE(dt, {
      const Grad<T> in = {static_cast<const T*>(grad), grad_stride};
      CR_LAUNCH(kKEmbeddingFew, s,
                (wide ? embedding_few_kernel<T, true> : embedding_few_kernel<T, false>)
                <<<(unsigned)ceil_div(vocab, kFewRows), 256, 0, s>>>(
                    tokens, index_bytes, (int)n, in, vocab, dim, (int)long_cols, out));
    });
    return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
  }
  const int64_t parts = n / kLong, part_warps = ceil_div(dim, kPartColumns);
  if (row_warps > kMaxBlocks / 2 / vocab || (parts > 0 && long_cols > kMaxBlocks / parts))
    return CR_ERR_UNSUPPORTED;
  char* at = past_status(ws);
  Sorted sorted;
  sorted.row_start = reinterpret_cast<int32_t*>(at);
  at += round256(((size_t)vocab + 1) * 4);
  sorted.order = reinterpret_cast<int32_t*>(at);
  at += round256((size_t)n * 4);
  sorted.part = reinterpret_cast<int32_t*>(at);
  at += round256((size_t)parts * 4);
  sorted.part_row = reinterpret_cast<int32_t*>(at);
  at += round256((size_t)parts * 4);
  float* sums = reinterpret_cast<float*>(at);
  const int rows = sort_rows(vocab);
  // Few tokens: fewer warps, whose counters take less time than the tokens
  // (1,037 tokens of 10,007 rows: 9.5 us with 8 warps, 11.0 with 32).
  const int sort_threads = n <= 8192 && rows <= 256 ? 256 : kSortThreads;
  const size_t smem = (size_t)rows * (sort_threads / 32) * 4;
  cudaError_t e = cudaFuncSetAttribute(token_sort_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSortRows * kSortWarps * 4);
  if (e != cudaSuccess) return CR_ERR_CUDA;
  CR_LAUNCH(kKTokenSort, s,
            token_sort_kernel<<<(unsigned)ceil_div(vocab, rows), sort_threads, smem, s>>>(
                tokens, index_bytes, n, vocab, rows, sorted));
  CR_MODEL_TYPE(dt, {
    const Grad<T> in = {static_cast<const T*>(grad), grad_stride};
    CR_LAUNCH(kKEmbeddingRows, s,
              (wide ? embedding_rows_kernel<T, true> : embedding_rows_kernel<T, false>)
              <<<(unsigned)ceil_div(parts * part_warps + vocab * row_warps, 8), 256, 0, s>>>(
                  in, sorted, parts * part_warps, part_warps, sums, vocab, dim, row_warps, out));
    if (parts > 0)
      CR_LAUNCH(kKEmbeddingLong, s,
                (wide ? embedding_long_kernel<T, true> : embedding_long_kernel<T, false>)
                <<<(unsigned)ceil_div(ceil_div(parts, kLongParts) * long_cols, 8), 256, 0, s>>>(
                    in, sorted, sums, parts, dim, long_cols, out));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
