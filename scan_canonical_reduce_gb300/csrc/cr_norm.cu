// Layer norm over rows and its gradient.
//
//   mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
//   n = (x - mean) rstd,  y = n w + b
//   g = dy w,  dx = rstd (g - sum(g) / D - n sum(g n) / D)
//   dw = sum over rows of dy n,  db = sum over rows of dy
//
// The mean is two numbers, the rounded one and the mean of what is left, so
// that a large mean takes nothing from n.
#include <algorithm>
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

struct Rows2 {
  int64_t bs, ts;
};

template <class T>
struct NormIn {
  int64_t rows, len, dim;
  float eps;
  const T* x;
  Rows2 xs;
  const float *w, *b;
};

__device__ __forceinline__ int64_t row_offset(int64_t r, int64_t len, Rows2 s) {
  int64_t t;
  const int64_t b = divide(r, len, t);
  return b * s.bs + t * s.ts;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s /= 2) v = __fadd_rn(v, __shfl_xor_sync(~0u, v, s));
  return v;
}

struct Stats {
  float mean, rest, rstd;
};

template <class T>
__device__ Stats row_stats(const T* x, int64_t dim, float eps, int lane) {
  float s = 0.0f;
  for (int64_t c = lane; c < dim; c += 32) s += to_f32(x[c]);
  Stats r;
  r.mean = warp_sum(s) / (float)dim;
  float d1 = 0.0f, d2 = 0.0f;
  for (int64_t c = lane; c < dim; c += 32) {
    const float d = to_f32(x[c]) - r.mean;
    d1 += d;
    d2 = fmaf(d, d, d2);
  }
  r.rest = warp_sum(d1) / (float)dim;
  const float var = fmaxf(warp_sum(d2) / (float)dim - r.rest * r.rest, 0.0f);
  r.rstd = 1.0f / sqrtf(var + eps);
  return r;
}

template <class T>
__global__ void __launch_bounds__(256)
layer_norm_kernel(NormIn<T> in, T* __restrict__ y, Rows2 ys, float* __restrict__ stats) {
  const int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (r >= in.rows) return;
  const T* x = in.x + row_offset(r, in.len, in.xs);
  const Stats st = row_stats(x, in.dim, in.eps, lane);
  T* yr = y + row_offset(r, in.len, ys);
  for (int64_t c = lane; c < in.dim; c += 32) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float w = in.w != nullptr ? in.w[c] : 1.0f, b = in.b != nullptr ? in.b[c] : 0.0f;
    yr[c] = from_f32<T>(fmaf(n, w, b));
  }
  if (stats != nullptr && lane == 0) {
    stats[3 * r] = st.mean;
    stats[3 * r + 1] = st.rest;
    stats[3 * r + 2] = st.rstd;
  }
}

// dx, and the row's statistics for the sums over rows
template <class T>
__global__ void __launch_bounds__(256)
layer_norm_backward_kernel(NormIn<T> in, const T* __restrict__ dy, Rows2 ds,
                           const float* __restrict__ stats, T* __restrict__ dx, Rows2 os,
                           float* __restrict__ kept) {
  const int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (r >= in.rows) return;
  const T* x = in.x + row_offset(r, in.len, in.xs);
  const T* d = dy + row_offset(r, in.len, ds);
  Stats st;
  if (stats != nullptr) st = {stats[3 * r], stats[3 * r + 1], stats[3 * r + 2]};
  else st = row_stats(x, in.dim, in.eps, lane);
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = lane; c < in.dim; c += 32) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float g = to_f32(d[c]) * (in.w != nullptr ? in.w[c] : 1.0f);
    s1 += g;
    s2 = fmaf(g, n, s2);
  }
  s1 = warp_sum(s1) / (float)in.dim;
  s2 = warp_sum(s2) / (float)in.dim;
  T* o = dx + row_offset(r, in.len, os);
  for (int64_t c = lane; c < in.dim; c += 32) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float g = to_f32(d[c]) * (in.w != nullptr ? in.w[c] : 1.0f);
    o[c] = from_f32<T>(st.rstd * fmaf(-n, s2, g - s1));
  }
  if (lane == 0) {
    kept[3 * r] = st.mean;
    kept[3 * r + 1] = st.rest;
    kept[3 * r + 2] = st.rstd;
  }
}

constexpr int kSumRows = 256;  // rows of a partial sum

template <class T>
__global__ void __launch_bounds__(256)
layer_norm_part_kernel(NormIn<T> in, const T* __restrict__ dy, Rows2 ds,
                       const float* __restrict__ stats, float* __restrict__ part) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= in.dim) return;
  for (int64_t p = blockIdx.y; p * kSumRows < in.rows; p += gridDim.y) {
    float dw = 0.0f, db = 0.0f;
    const int64_t end = min(in.rows, (p + 1) * kSumRows);
    for (int64_t r = p * kSumRows; r < end; ++r) {
      const float x = to_f32(in.x[row_offset(r, in.len, in.xs) + c]);
      const float d = to_f32(dy[row_offset(r, in.len, ds) + c]);
      const float n = ((x - stats[3 * r]) - stats[3 * r + 1]) * stats[3 * r + 2];
      dw = fmaf(d, n, dw);
      db += d;
    }
    part[2 * p * in.dim + c] = dw;
    part[(2 * p + 1) * in.dim + c] = db;
  }
}

__global__ void __launch_bounds__(256)
layer_norm_sum_kernel(const float* __restrict__ part, int64_t parts, int64_t dim,
                      float* __restrict__ dw, float* __restrict__ db) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= dim) return;
  float w = 0.0f, b = 0.0f;
  for (int64_t p = 0; p < parts; ++p) {
    w += part[2 * p * dim + c];
    b += part[(2 * p + 1) * dim + c];
  }
  if (dw != nullptr) dw[c] = w;
  if (db != nullptr) db[c] = b;
}

template <class T>
NormIn<T> norm_in(const cr_layer_norm_args* a) {
  return {a->batch * a->len, a->len, a->dim, a->eps, static_cast<const T*>(a->x),
          {a->x_batch_stride, a->x_time_stride}, a->weight, a->bias};
}

bool rows_fit(const cr_layer_norm_args* a, int64_t bs, int64_t ts) {
  return (a->len <= 1 || ts >= a->dim) && (a->batch <= 1 || bs >= a->dim);
}

cr_status check_norm(const cr_layer_norm_args* a) {
  if (a == nullptr) return CR_ERR_INVALID_ARG;
  const size_t es = model_esize(a->dt);
  if (es == 0 || a->batch < 0 || a->len < 0 || a->dim < 0 || !(a->eps >= 0.0f) ||
      a->x_batch_stride < 0 || a->x_time_stride < 0)
    return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->len > 0 && a->dim > 0 && a->x == nullptr) return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(a->x, es) || !ptr_aligned(a->weight, 4) || !ptr_aligned(a->bias, 4))
    return CR_ERR_INVALID_ARG;
  if (a->len > 0 && a->batch > kMaxBlocks / a->len) return CR_ERR_UNSUPPORTED;
  return CR_OK;
}

}  // namespace
}  // namespace cr

extern "C" {

cr_status cr_layer_norm(const cr_layer_norm_args* a, void* y, int64_t y_batch_stride,
                        int64_t y_time_stride, float* stats, void* stream) {
  using namespace cr;
  const cr_status ok = check_norm(a);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt);
  if (y_batch_stride < 0 || y_time_stride < 0) return CR_ERR_INVALID_ARG;
  const int64_t rows = a->batch * a->len;
  if (rows == 0 || a->dim == 0) return CR_OK;
  if (y == nullptr || !rows_fit(a, y_batch_stride, y_time_stride) || !ptr_aligned(y, es) ||
      !ptr_aligned(stats, 4) || overwrites({y, stats}, {a->x, a->weight, a->bias}))
    return CR_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    CR_LAUNCH(kKLayerNorm, s,
              layer_norm_kernel<T><<<(unsigned)ceil_div(rows, 8), 256, 0, s>>>(
                  norm_in<T>(a), static_cast<T*>(y), Rows2{y_batch_stride, y_time_stride},
                  stats));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

size_t cr_layer_norm_backward_workspace_bytes(int64_t batch, int64_t len, int64_t dim) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || (len > 0 && batch > kMaxBlocks / len)) return 0;
  const int64_t rows = batch * len;
  return round256((size_t)rows * 12) + round256((size_t)ceil_div(rows, kSumRows) * dim * 8) +
         kStatusBytes;
}

cr_status cr_layer_norm_backward(const cr_layer_norm_args* a, const cr_layer_norm_grads* g,
                                 void* ws, size_t ws_bytes, void* stream) {
  using namespace cr;
  const cr_status ok = check_norm(a);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt);
  if (g == nullptr || g->dy_batch_stride < 0 || g->dy_time_stride < 0 ||
      g->dx_batch_stride < 0 || g->dx_time_stride < 0)
    return CR_ERR_INVALID_ARG;
  const int64_t rows = a->batch * a->len;
  if (a->dim == 0) return CR_OK;
  if (rows > 0 && (g->dy == nullptr || g->dx == nullptr ||
                   !rows_fit(a, g->dx_batch_stride, g->dx_time_stride)))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(g->dy, es) || !ptr_aligned(g->dx, es) || !ptr_aligned(g->stats, 4) ||
      !ptr_aligned(g->dweight, 4) || !ptr_aligned(g->dbias, 4) ||
      overwrites({g->dx, g->dweight, g->dbias}, {a->x, a->weight, a->bias, g->dy, g->stats}))
    return CR_ERR_INVALID_ARG;
  const size_t need = cr_layer_norm_backward_workspace_bytes(a->batch, a->len, a->dim);
  if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < need) return CR_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* at = past_status(ws);
  float* kept = reinterpret_cast<float*>(at);
  float* part = reinterpret_cast<float*>(at + round256((size_t)rows * 12));
  const int64_t parts = ceil_div(rows, kSumRows), cols = ceil_div(a->dim, 256);
  if (cols > kMaxBlocks) return CR_ERR_UNSUPPORTED;
  const Rows2 ds = {g->dy_batch_stride, g->dy_time_stride};
  CR_MODEL_TYPE(a->dt, {
    const T* dy = static_cast<const T*>(g->dy);
    if (rows > 0) {
      CR_LAUNCH(kKLayerNormBackward, s,
                layer_norm_backward_kernel<T><<<(unsigned)ceil_div(rows, 8), 256, 0, s>>>(
                    norm_in<T>(a), dy, ds, g->stats, static_cast<T*>(g->dx),
                    Rows2{g->dx_batch_stride, g->dx_time_stride}, kept));
      CR_LAUNCH(kKLayerNormSum, s,
                layer_norm_part_kernel<T>
                <<<dim3((unsigned)cols, (unsigned)std::min<int64_t>(parts, 65535)), 256, 0, s>>>(
                    norm_in<T>(a), dy, ds, kept, part));
    }
    if (g->dweight != nullptr || g->dbias != nullptr)
      CR_LAUNCH(kKLayerNormSum, s,
                layer_norm_sum_kernel<<<(unsigned)cols, 256, 0, s>>>(part, parts, a->dim,
                                                                     g->dweight, g->dbias));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
