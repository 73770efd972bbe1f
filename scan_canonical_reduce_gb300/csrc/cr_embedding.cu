// Embedding lookup and its gradient.
//
//   out[i] = scale * table[tokens[i]]
//   dW[v]  = scale * tree(grad[p] : tokens[p] == v, p ascending)
//
// The gradient is a reduction per token, and takes the library's expression
// for one: the shift-reduce tree over the rows in order. Equal tokens are
// brought together by a stable counting sort (integers only, so its result is
// unique), then every row of the table is one tree.
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

// ------------------------------------------------------------- lookup
// A block covers blockDim.y tokens; the threads of a row walk its columns.
template <class T, int V>
__global__ void __launch_bounds__(256)
embedding_kernel(const void* __restrict__ tokens, int index_bytes, int64_t n,
                 const T* __restrict__ table, int64_t vocab, int64_t dim, int64_t row_stride,
                 float scale, T* __restrict__ out, int64_t out_stride, bool wide) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (i >= n) return;
  const int64_t v = load_index(tokens, index_bytes, i);
  const bool real = v >= 0 && v < vocab;
  const T* src = table + (real ? v : 0) * row_stride;
  T* dst = out + i * out_stride;
  for (int64_t c = (int64_t)threadIdx.x * V; c < dim; c += (int64_t)blockDim.x * V) {
    const int have = (int)min((int64_t)V, dim - c);
    const bool w = wide && have == V;
    float f[V];
    if (real) {
      load_f32<T, V>(src + c, w, have, f);
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = f[k] * scale;
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = 0.0f;
    }
    store_f32<T, V>(dst + c, w, have, f);
  }
}

// --------------------------------------------------------------- sort
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRows = 1024;  // most rows a block sorts: 128 KB of counters

// Stable counting sort of the positions by token. Block j owns the rows
// [j R, (j+1) R) and reads every token, so that it needs nothing of another
// block: the number of smaller tokens is where its part of `order` begins.
// Warp w owns the w-th contiguous part of the positions in both sweeps; its
// counters are its own, and within 32 positions equal tokens are ranked by
// lane, so the order is that of the positions.
__global__ void __launch_bounds__(kSortThreads)
token_sort_kernel(const void* __restrict__ tokens, int index_bytes, int64_t n, int64_t vocab,
                  int rows_per_block, int32_t* __restrict__ row_start,
                  int32_t* __restrict__ order) {
  extern __shared__ int32_t count[];  // [warp][row], then cursors
  __shared__ int32_t warp_total[kSortWarps];
  __shared__ int32_t base_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t lo = (int64_t)blockIdx.x * rows_per_block;
  const int64_t hi = min(vocab, lo + rows_per_block);
  const int R = (int)(hi - lo);
  for (int k = tid; k < R * kSortWarps; k += kSortThreads) count[k] = 0;
  if (tid == 0) base_s = 0;
  __syncthreads();

  const int64_t part = ((n + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t p0 = min(n, warp * part), p1 = min(n, p0 + part);
  int32_t* mine = count + warp * R;
  int32_t below = 0;
  for (int64_t p = p0 + lane; p < p1; p += 32) {
    const int64_t v = load_index(tokens, index_bytes, p);
    if (v >= 0 && v < lo) ++below;
    if (v >= lo && v < hi) atomicAdd(&mine[v - lo], 1);
  }
  below = __reduce_add_sync(~0u, below);
  if (lane == 0) atomicAdd(&base_s, below);
  __syncthreads();
  const int32_t base = base_s;

  // Exclusive prefix over rows of the rows' totals, and within a row over
  // warps: thread r takes row r (R <= 1024).
  int32_t total = 0;
  if (tid < R)
    for (int w = 0; w < kSortWarps; ++w) total += count[w * R + tid];
  int32_t incl = total;
  for (int s = 1; s < 32; s *= 2) {
    const int32_t o = __shfl_up_sync(~0u, incl, s);
    if (lane >= s) incl += o;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  int32_t before = base;
  for (int w = 0; w < warp; ++w) before += warp_total[w];
  int32_t start = before + incl - total;
  if (tid < R) {
    row_start[lo + tid] = start;
    if (lo + tid == vocab - 1) row_start[vocab] = start + total;
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t c = count[w * R + tid];
      count[w * R + tid] = start;
      start += c;
    }
  }
  __syncthreads();

  for (int64_t q = p0; q < p1; q += 32) {
    const int64_t p = q + lane;
    const int64_t v = p < p1 ? load_index(tokens, index_bytes, p) : -1;
    const bool in = v >= lo && v < hi;
    const uint32_t any = __ballot_sync(~0u, in);
    if (any == 0) continue;
    if (in) {
      const int r = (int)(v - lo);
      const uint32_t same = __match_any_sync(any, r);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int32_t at = mine[r];
      __syncwarp(any);
      if (rank == 0) mine[r] = at + __popc(same);
      order[at + rank] = (int32_t)p;
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------- row trees
constexpr int kRowThreads = 256;
constexpr int kRowGroup = 8;    // rows read at a time
constexpr int kRowLevels = 32;  // of the tree above a group

// One warp: one row of the table, 128 columns (4 a lane). Groups of 8 rows
// are perfect trees in registers; their values go through the shift-reduce
// stack (a binary counter in local memory, one access a group).
template <class T>
__global__ void __launch_bounds__(kRowThreads)
embedding_rows_kernel(const T* __restrict__ grad, int64_t grad_stride, bool wide,
                      const int32_t* __restrict__ row_start, const int32_t* __restrict__ order,
                      int64_t vocab, int64_t dim, int64_t col_blocks, float scale,
                      bool accumulate, float* __restrict__ dw, int64_t dw_stride, bool wide_dw) {
  const int64_t v = blockIdx.x / col_blocks;
  const int64_t c = (blockIdx.x % col_blocks * kRowThreads + threadIdx.x) * 4;
  if (c >= dim) return;
  const int have = (int)min((int64_t)4, dim - c);
  const bool w = wide && have == 4, wd = wide_dw && have == 4;
  const int32_t first = row_start[v], last = row_start[v + 1];
  if (first == last && accumulate) return;

  float stack[kRowLevels][4];
  uint32_t blocks = 0;  // full groups so far: the counter of the stack
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int32_t p = first;
  for (; p + kRowGroup <= last; p += kRowGroup) {
    float g[kRowGroup][4];
#pragma unroll
    for (int k = 0; k < kRowGroup; ++k)
      load_f32<T, 4>(grad + order[p + k] * grad_stride + c, w, have, g[k]);
#pragma unroll
    for (int s = 1; s < kRowGroup; s *= 2)
#pragma unroll
      for (int k = 0; k < kRowGroup; k += 2 * s)
#pragma unroll
        for (int j = 0; j < 4; ++j) g[k][j] = add_rn(g[k][j], g[k + s][j]);
    int lv = 0;
    for (; (blocks >> lv) & 1u; ++lv)
#pragma unroll
      for (int j = 0; j < 4; ++j) g[0][j] = add_rn(stack[lv][j], g[0][j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) stack[lv][j] = g[0][j];
    ++blocks;
  }
  // The tail (fewer than 8 rows): its own stack of three levels, folded from
  // the right, then the groups' stack, smallest block first.
  bool has = false;
  const int tail = last - p;
  if (tail > 0) {
    float t[kRowGroup - 1][4];
#pragma unroll
    for (int k = 0; k < kRowGroup - 1; ++k)
      if (k < tail) load_f32<T, 4>(grad + order[p + k] * grad_stride + c, w, have, t[k]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      RegStack<float, 3> st;
      st.reset();
#pragma unroll
      for (int k = 0; k < kRowGroup - 1; ++k)
        if (k < tail) st.push(t[k][j], 0);
      bool h = false;
      float a = 0.0f;
      h = st.fold_onto(a, h);
      acc[j] = a;
    }
    has = true;
  }
  for (int lv = 0; (blocks >> lv) != 0; ++lv) {
    if ((blocks >> lv) & 1u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = has ? add_rn(stack[lv][j], acc[j]) : stack[lv][j];
      has = true;
    }
  }
  float* dst = dw + v * dw_stride + c;
  if (has) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = acc[j] * scale;
    if (accumulate) {
      float old[4];
      load_f32<float, 4>(dst, wd, have, old);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = add_rn(old[j], acc[j]);
    }
  }
  store_f32<float, 4>(dst, wd, have, acc);
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
  if (tokens == nullptr || out == nullptr || (vocab > 0 && table == nullptr) || out == table)
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
              embedding_kernel<T, V><<<(unsigned)blocks, block, 0, s>>>(
                  tokens, index_bytes, n, static_cast<const T*>(table), vocab, dim, row_stride,
                  scale, static_cast<T*>(out), out_stride, wide));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

size_t cr_embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  using namespace cr;
  if (n < 0 || vocab < 0 || dim < 0 || n > INT32_MAX || vocab > INT32_MAX) return 0;
  return round256(((size_t)vocab + 1) * 4) + round256((size_t)n * 4) + 256;
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
  if (vocab > 0 && dim > 0 && (dw == nullptr || dw == grad)) return CR_ERR_INVALID_ARG;
  if ((tokens && !ptr_aligned(tokens, index_bytes)) || (grad && !ptr_aligned(grad, es)) ||
      (dw && !ptr_aligned(dw, 4)))
    return CR_ERR_INVALID_ARG;
  if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < need) return CR_ERR_WORKSPACE;
  if (vocab == 0 || dim == 0) return CR_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t col_blocks = ceil_div(dim, kRowThreads * 4);
  if (col_blocks > kMaxBlocks / vocab) return CR_ERR_UNSUPPORTED;
  int32_t* row_start = static_cast<int32_t*>(ws);
  int32_t* order = reinterpret_cast<int32_t*>(static_cast<char*>(ws) +
                                              round256(((size_t)vocab + 1) * 4));
  const int rows = sort_rows(vocab);
  const size_t smem = (size_t)rows * kSortWarps * 4;
  cudaError_t e = cudaFuncSetAttribute(token_sort_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSortRows * kSortWarps * 4);
  if (e != cudaSuccess) return CR_ERR_CUDA;
  CR_LAUNCH(kKTokenSort, s,
            token_sort_kernel<<<(unsigned)ceil_div(vocab, rows), kSortThreads, smem, s>>>(
                tokens, index_bytes, n, vocab, rows, row_start, order));
  const bool wide = rows_aligned(grad, grad_stride, 0, es, 4 * es);
  const bool wide_dw = rows_aligned(dw, dw_stride, 0, 4, 16);
  CR_MODEL_TYPE(dt, {
    CR_LAUNCH(kKEmbeddingRows, s,
              embedding_rows_kernel<T><<<(unsigned)(vocab * col_blocks), kRowThreads, 0, s>>>(
                  static_cast<const T*>(grad), grad_stride, wide, row_start, order, vocab, dim,
                  col_blocks, scale, accumulate != 0, dw, dw_stride, wide_dw));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
