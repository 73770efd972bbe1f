// Depthwise causal convolution over time, its gradient, and its single-token
// form.
//
//   pre[t] = bias + sum_{k<K} w[k] x[t-(K-1)+k],   y[t] = act(pre[t])
//   dpre[t] = dy[t] act'(pre[t])
//   dx[p] = sum_{k<K} w[k] dpre[p+(K-1)-k],  dw[k] = sum_t dpre[t] x[t-(K-1)+k]
//
// A thread takes V neighbouring channels and a run of time steps, and keeps
// the last K inputs (backward: and the last K of dpre) in registers, so that
// each input is read once, plus K-1 steps of halo a run.
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

constexpr int kConvThreads = 128;
constexpr int kV = 4;  // channels a thread

struct ConvShape {
  int64_t batch, len, dim;
  int64_t runs;       // runs of kRun steps a sequence (at least 1)
  int64_t col_blocks; // blocks along the channels
};
constexpr int kRun = 64;

ConvShape conv_shape(int64_t batch, int64_t len, int64_t dim) {
  ConvShape c;
  c.batch = batch;
  c.len = len;
  c.dim = dim;
  c.runs = len > 0 ? ceil_div(len, kRun) : 1;
  c.col_blocks = ceil_div(dim, kConvThreads * kV);
  return c;
}

// What every kernel of a (batch, time, channel) call reads.
template <class T>
struct ConvIn {
  const T* x;
  int64_t bs, ts;
  const float* weight;
  const float* bias;
  const T* state;
  const void* lengths;
  int index_bytes;
  bool silu, wide, wide_state;
};

// Input at extended time t (t < 0: the state's) of channels c .. c + have.
template <class T, int K>
__device__ __forceinline__ void conv_input(const ConvIn<T>& in, const ConvShape& sh, int64_t b,
                                           int64_t t, int64_t c, int have, float (&f)[kV]) {
  if (t >= 0) {
    load_f32<T, kV>(in.x + b * in.bs + t * in.ts + c, in.wide && have == kV, have, f);
  } else if (in.state != nullptr) {
    load_f32<T, kV>(in.state + (b * (K - 1) + (K - 1 + t)) * sh.dim + c,
                    in.wide_state && have == kV, have, f);
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) f[j] = 0.0f;
  }
}

template <int K>
__device__ __forceinline__ void conv_weights(const float* weight, const float* bias, int64_t c,
                                             int have, float (&w)[K][kV], float (&b0)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    b0[j] = (bias != nullptr && j < have) ? bias[c + j] : 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][j] = j < have ? weight[(c + j) * K + k] : 0.0f;
  }
}

template <class T, int K>
__global__ void __launch_bounds__(kConvThreads)
causal_conv_kernel(ConvIn<T> in, ConvShape sh, T* __restrict__ y, int64_t ybs, int64_t yts,
                   bool wide_y, T* __restrict__ final_state) {
  int64_t i = blockIdx.x;
  const int64_t c = (i % sh.col_blocks * kConvThreads + threadIdx.x) * kV;
  i /= sh.col_blocks;
  const int64_t run = i % sh.runs, b = i / sh.runs;
  if (c >= sh.dim) return;
  const int have = (int)min((int64_t)kV, sh.dim - c);
  const int64_t len = sequence_length(in.lengths, in.index_bytes, b, sh.len);
  const int64_t t0 = run * kRun, t1 = min(sh.len, t0 + kRun);
  const bool wy = wide_y && have == kV;

  if (t0 < len) {
    float w[K][kV], b0[kV], win[K][kV];
    conv_weights<K>(in.weight, in.bias, c, have, w, b0);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      conv_input<T, K>(in, sh, b, t0 - (K - 1) + k, c, have, win[k + 1]);
    for (int64_t t = t0; t < min(t1, len); ++t) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j) win[k][j] = win[k + 1][j];
      conv_input<T, K>(in, sh, b, t, c, have, win[K - 1]);
      float o[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        float p = b0[j];
#pragma unroll
        for (int k = 0; k < K; ++k) p = fmaf(w[k][j], win[k][j], p);
        o[j] = in.silu ? p * sigmoid(p) : p;
      }
      store_f32<T, kV>(y + b * ybs + t * yts + c, wy, have, o);
    }
  }
  const float zero[kV] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t t = max(t0, len); t < t1; ++t)
    store_f32<T, kV>(y + b * ybs + t * yts + c, wy, have, zero);
  if (run == 0 && final_state != nullptr) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      float f[kV];
      conv_input<T, K>(in, sh, b, len - (K - 1) + j, c, have, f);
      store_f32<T, kV>(final_state + (b * (K - 1) + j) * sh.dim + c, in.wide_state && have == kV,
                       have, f);
    }
  }
}

template <class T>
struct ConvBack {
  const T* dy;
  int64_t dybs, dyts;
  const T* dfinal;
  T* dx;
  int64_t dxbs, dxts;
  T* dstate;
  float* part;  // [batch x runs][dim][K + 1]: dw, then dbias
  bool wide_dx;
};

// A run computes dpre for its own steps and the K-1 after them; it writes
// dx of its own steps (run 0: of the state's too) and the sums of
// dpre x and dpre over its own steps.
template <class T, int K>
__global__ void __launch_bounds__(kConvThreads)
causal_conv_backward_kernel(ConvIn<T> in, ConvShape sh, ConvBack<T> g) {
  int64_t i = blockIdx.x;
  const int64_t c = (i % sh.col_blocks * kConvThreads + threadIdx.x) * kV;
  i /= sh.col_blocks;
  const int64_t run = i % sh.runs, b = i / sh.runs;
  if (c >= sh.dim) return;
  const int have = (int)min((int64_t)kV, sh.dim - c);
  const int64_t len = sequence_length(in.lengths, in.index_bytes, b, sh.len);
  const int64_t t0 = run * kRun, t1 = min(sh.len, t0 + kRun);

  float w[K][kV], b0[kV], win[K][kV], dp[K][kV], dw[K][kV], db[kV];
  conv_weights<K>(in.weight, in.bias, c, have, w, b0);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < kV; ++j) win[k][j] = dp[k][j] = dw[k][j] = 0.0f;
#pragma unroll
  for (int j = 0; j < kV; ++j) db[j] = 0.0f;
  if (t0 < len || run == 0) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      conv_input<T, K>(in, sh, b, t0 - (K - 1) + k, c, have, win[k + 1]);
    // after step t the window dp holds dpre[t-K+1 .. t], which completes
    // dx at p = t - K + 1
    for (int64_t t = t0; t < t1 + K - 1; ++t) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          win[k][j] = win[k + 1][j];
          dp[k][j] = dp[k + 1][j];
        }
      if (t < len) {
        float d[kV];
        conv_input<T, K>(in, sh, b, t, c, have, win[K - 1]);
        load_f32<T, kV>(g.dy + b * g.dybs + t * g.dyts + c, in.wide && have == kV, have, d);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          float p = b0[j];
#pragma unroll
          for (int k = 0; k < K; ++k) p = fmaf(w[k][j], win[k][j], p);
          if (in.silu) {
            const float s = sigmoid(p);
            d[j] = d[j] * (s * fmaf(p, 1.0f - s, 1.0f));
          }
          dp[K - 1][j] = d[j];
          if (t < t1) {
            db[j] += d[j];
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][j] = fmaf(d[j], win[k][j], dw[k][j]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) dp[K - 1][j] = 0.0f;
      }
      const int64_t p = t - (K - 1);
      if (p < t0 && run != 0) continue;  // the run before writes it
      float o[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        o[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) o[j] = fmaf(w[k][j], dp[K - 1 - k][j], o[j]);
      }
      if (g.dfinal != nullptr && p >= len - (K - 1) && p < len) {
        float f[kV];
        load_f32<T, kV>(g.dfinal + (b * (K - 1) + (p - (len - (K - 1)))) * sh.dim + c,
                        in.wide_state && have == kV, have, f);
#pragma unroll
        for (int j = 0; j < kV; ++j) o[j] += f[j];
      }
      if (p >= 0) {
        if (g.dx != nullptr && p < sh.len)
          store_f32<T, kV>(g.dx + b * g.dxbs + p * g.dxts + c, g.wide_dx && have == kV, have, o);
      } else if (g.dstate != nullptr) {
        store_f32<T, kV>(g.dstate + (b * (K - 1) + (K - 1 + p)) * sh.dim + c,
                         in.wide_state && have == kV, have, o);
      }
    }
  } else if (g.dx != nullptr) {
    const float zero[kV] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t t = t0; t < t1; ++t)
      store_f32<T, kV>(g.dx + b * g.dxbs + t * g.dxts + c, g.wide_dx && have == kV, have, zero);
  }
  float* part = g.part + ((b * sh.runs + run) * sh.dim + c) * (K + 1);
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    if (j < have) {
#pragma unroll
      for (int k = 0; k < K; ++k) part[j * (K + 1) + k] = dw[k][j];
      part[j * (K + 1) + K] = db[j];
    }
  }
}

// Sums the runs' partials in order: thread i takes one (channel, tap).
__global__ void __launch_bounds__(kConvThreads)
causal_conv_sum_kernel(const float* __restrict__ part, int64_t parts, int64_t dim, int K,
                       float* __restrict__ dweight, float* __restrict__ dbias) {
  const int64_t n = dim * (K + 1);
  const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int64_t p = 0; p < parts; ++p) s += part[p * n + i];
  const int64_t d = i / (K + 1);
  const int k = (int)(i % (K + 1));
  if (k < K) dweight[d * K + k] = s;
  else if (dbias != nullptr) dbias[d] = s;
}

template <class T, int K>
__global__ void __launch_bounds__(kConvThreads)
causal_conv_step_kernel(const T* __restrict__ x, int64_t x_stride, T* __restrict__ state,
                        int64_t state_rows, const void* __restrict__ slots, int index_bytes,
                        const float* __restrict__ weight, const float* __restrict__ bias,
                        bool silu, int64_t dim, int64_t col_blocks, bool wide, bool wide_state,
                        T* __restrict__ y, int64_t y_stride) {
  const int64_t b = blockIdx.x / col_blocks;
  const int64_t c = (blockIdx.x % col_blocks * kConvThreads + threadIdx.x) * kV;
  if (c >= dim) return;
  const int have = (int)min((int64_t)kV, dim - c);
  const bool full = have == kV;
  const int64_t row = slots != nullptr ? load_index(slots, index_bytes, b) : b;
  float o[kV] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (row >= 0 && row < state_rows) {
    float w[K][kV], b0[kV], win[K][kV];
    conv_weights<K>(weight, bias, c, have, w, b0);
    T* st = state + row * (K - 1) * dim + c;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load_f32<T, kV>(st + k * dim, wide_state && full, have, win[k]);
    load_f32<T, kV>(x + b * x_stride + c, wide && full, have, win[K - 1]);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      float p = b0[j];
#pragma unroll
      for (int k = 0; k < K; ++k) p = fmaf(w[k][j], win[k][j], p);
      o[j] = silu ? p * sigmoid(p) : p;
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      store_f32<T, kV>(st + k * dim, wide_state && full, have, win[k + 1]);
  }
  store_f32<T, kV>(y + b * y_stride + c, wide && full, have, o);
}

// The checks that the forward and the backward call share.
cr_status check_conv(const cr_causal_conv_args* a) {
  if (a == nullptr) return CR_ERR_INVALID_ARG;
  const size_t es = model_esize(a->dt);
  if (es == 0 || a->batch < 0 || a->len < 0 || a->dim < 0 || a->x_batch_stride < 0 ||
      a->x_time_stride < 0)
    return CR_ERR_INVALID_ARG;
  if (a->activation != CR_ACT_NONE && a->activation != CR_ACT_SILU) return CR_ERR_INVALID_ARG;
  if (a->width < 1) return CR_ERR_INVALID_ARG;
  if (a->width < 2 || a->width > 4) return CR_ERR_UNSUPPORTED;
  if (a->lengths != nullptr &&
      (!index_width_ok(a->index_bytes) || !ptr_aligned(a->lengths, a->index_bytes)))
    return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->dim > 0 && (a->weight == nullptr || (a->len > 0 && a->x == nullptr)))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(a->x, es) || !ptr_aligned(a->state, es) || !ptr_aligned(a->weight, 4) ||
      !ptr_aligned(a->bias, 4))
    return CR_ERR_INVALID_ARG;
  const ConvShape sh = conv_shape(a->batch, a->len, a->dim);
  if (a->batch > 0 && a->dim > 0 &&
      (double)sh.batch * (double)sh.runs * (double)sh.col_blocks > (double)kMaxBlocks)
    return CR_ERR_UNSUPPORTED;
  return CR_OK;
}

template <class T>
ConvIn<T> conv_in(const cr_causal_conv_args* a, bool wide, bool wide_state) {
  ConvIn<T> in;
  in.x = static_cast<const T*>(a->x);
  in.bs = a->x_batch_stride;
  in.ts = a->x_time_stride;
  in.weight = a->weight;
  in.bias = a->bias;
  in.state = static_cast<const T*>(a->state);
  in.lengths = a->lengths;
  in.index_bytes = a->index_bytes;
  in.silu = a->activation == CR_ACT_SILU;
  in.wide = wide;
  in.wide_state = wide_state;
  return in;
}

// Runs BODY with K bound to the width.
#define CR_CONV_WIDTH(WIDTH, ...)                            \
  switch (WIDTH) {                                           \
    case 2: { constexpr int K = 2; __VA_ARGS__; break; }     \
    case 3: { constexpr int K = 3; __VA_ARGS__; break; }     \
    default: { constexpr int K = 4; __VA_ARGS__; break; }    \
  }

}  // namespace
}  // namespace cr

extern "C" {

cr_status cr_causal_conv(const cr_causal_conv_args* a, void* y, int64_t y_batch_stride,
                         int64_t y_time_stride, void* final_state, void* stream) {
  using namespace cr;
  const cr_status ok = check_conv(a);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt);
  if (y_batch_stride < 0 || y_time_stride < 0) return CR_ERR_INVALID_ARG;
  if (a->batch == 0 || a->dim == 0) return CR_OK;
  if (a->len > 0 && (y == nullptr || y == a->x || (a->len > 1 && y_time_stride < a->dim) ||
                     (a->batch > 1 && y_batch_stride < a->dim)))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(y, es) || !ptr_aligned(final_state, es)) return CR_ERR_INVALID_ARG;
  if (a->len == 0 && final_state == nullptr) return CR_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ConvShape sh = conv_shape(a->batch, a->len, a->dim);
  const unsigned blocks = (unsigned)(sh.batch * sh.runs * sh.col_blocks);
  const bool wide = rows_aligned(a->x, a->x_batch_stride, a->x_time_stride, es, kV * es);
  const bool wide_y = rows_aligned(y, y_batch_stride, y_time_stride, es, kV * es);
  const bool wide_state = rows_aligned(a->state, a->dim, a->dim, es, kV * es) &&
                          rows_aligned(final_state, a->dim, a->dim, es, kV * es);
  CR_MODEL_TYPE(a->dt, CR_CONV_WIDTH(a->width, {
    CR_LAUNCH(kKCausalConv, s,
              causal_conv_kernel<T, K><<<blocks, kConvThreads, 0, s>>>(
                  conv_in<T>(a, wide, wide_state), sh, static_cast<T*>(y), y_batch_stride,
                  y_time_stride, wide_y, static_cast<T*>(final_state)));
  }));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

size_t cr_causal_conv_backward_workspace_bytes(int64_t batch, int64_t len, int64_t dim,
                                               int32_t width) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || width < 1) return 0;
  const ConvShape sh = conv_shape(batch, len, dim);
  return round256((size_t)(batch * sh.runs) * (size_t)dim * (width + 1) * 4) + 256;
}

cr_status cr_causal_conv_backward(const cr_causal_conv_args* a, const cr_causal_conv_grads* g,
                                  void* ws, size_t ws_bytes, void* stream) {
  using namespace cr;
  const cr_status ok = check_conv(a);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt);
  if (g == nullptr || g->dy_batch_stride < 0 || g->dy_time_stride < 0 ||
      g->dx_batch_stride < 0 || g->dx_time_stride < 0)
    return CR_ERR_INVALID_ARG;
  if (a->dim == 0) return CR_OK;
  if (g->dweight == nullptr) return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->len > 0) {
    if (g->dy == nullptr || (g->dx != nullptr && (g->dx == g->dy || g->dx == a->x)))
      return CR_ERR_INVALID_ARG;
    if (g->dx != nullptr && ((a->len > 1 && g->dx_time_stride < a->dim) ||
                             (a->batch > 1 && g->dx_batch_stride < a->dim)))
      return CR_ERR_INVALID_ARG;
  }
  if (!ptr_aligned(g->dy, es) || !ptr_aligned(g->dx, es) || !ptr_aligned(g->dfinal, es) ||
      !ptr_aligned(g->dstate, es) || !ptr_aligned(g->dweight, 4) || !ptr_aligned(g->dbias, 4))
    return CR_ERR_INVALID_ARG;
  const size_t need = cr_causal_conv_backward_workspace_bytes(a->batch, a->len, a->dim, a->width);
  if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < need) return CR_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ConvShape sh = conv_shape(a->batch, a->len, a->dim);
  if (a->batch > 0) {
    const unsigned blocks = (unsigned)(sh.batch * sh.runs * sh.col_blocks);
    const bool wide = rows_aligned(a->x, a->x_batch_stride, a->x_time_stride, es, kV * es) &&
                      rows_aligned(g->dy, g->dy_batch_stride, g->dy_time_stride, es, kV * es);
    const bool wide_dx = rows_aligned(g->dx, g->dx_batch_stride, g->dx_time_stride, es, kV * es);
    const bool wide_state = rows_aligned(a->state, a->dim, a->dim, es, kV * es) &&
                            rows_aligned(g->dstate, a->dim, a->dim, es, kV * es) &&
                            rows_aligned(g->dfinal, a->dim, a->dim, es, kV * es);
    CR_MODEL_TYPE(a->dt, CR_CONV_WIDTH(a->width, {
      ConvBack<T> gb;
      gb.dy = static_cast<const T*>(g->dy);
      gb.dybs = g->dy_batch_stride;
      gb.dyts = g->dy_time_stride;
      gb.dfinal = static_cast<const T*>(g->dfinal);
      gb.dx = static_cast<T*>(g->dx);
      gb.dxbs = g->dx_batch_stride;
      gb.dxts = g->dx_time_stride;
      gb.dstate = static_cast<T*>(g->dstate);
      gb.part = static_cast<float*>(ws);
      gb.wide_dx = wide_dx;
      CR_LAUNCH(kKCausalConvBackward, s,
                causal_conv_backward_kernel<T, K><<<blocks, kConvThreads, 0, s>>>(
                    conv_in<T>(a, wide, wide_state), sh, gb));
    }));
    if (cudaGetLastError() != cudaSuccess) return CR_ERR_CUDA;
  }
  const int64_t n = a->dim * (a->width + 1);
  CR_LAUNCH(kKCausalConvSum, s,
            causal_conv_sum_kernel<<<(unsigned)ceil_div(n, kConvThreads), kConvThreads, 0, s>>>(
                static_cast<const float*>(ws), a->batch * sh.runs, a->dim, a->width, g->dweight,
                g->dbias));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

cr_status cr_causal_conv_step(const void* x, int64_t x_stride, void* state, int64_t state_rows,
                              const void* slots, int32_t index_bytes, const float* weight,
                              const float* bias, int32_t activation, int64_t batch, int64_t dim,
                              int32_t width, cr_dtype dt, void* y, int64_t y_stride,
                              void* stream) {
  using namespace cr;
  const size_t es = model_esize(dt);
  if (es == 0 || batch < 0 || dim < 0 || state_rows < 0 || x_stride < 0 || width < 1)
    return CR_ERR_INVALID_ARG;
  if (activation != CR_ACT_NONE && activation != CR_ACT_SILU) return CR_ERR_INVALID_ARG;
  if (width < 2 || width > 4) return CR_ERR_UNSUPPORTED;
  if (slots != nullptr ? !index_width_ok(index_bytes) || !ptr_aligned(slots, index_bytes)
                       : state_rows < batch)
    return CR_ERR_INVALID_ARG;
  if (batch == 0 || dim == 0) return CR_OK;
  if (x == nullptr || weight == nullptr || y == nullptr || y == x || y == state || x == state ||
      (state == nullptr && state_rows > 0) || (batch > 1 && y_stride < dim) || y_stride < 0)
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(x, es) || !ptr_aligned(state, es) || !ptr_aligned(y, es) ||
      !ptr_aligned(weight, 4) || !ptr_aligned(bias, 4))
    return CR_ERR_INVALID_ARG;
  const int64_t col_blocks = ceil_div(dim, kConvThreads * kV);
  if (col_blocks > kMaxBlocks / batch) return CR_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = rows_aligned(x, x_stride, 0, es, kV * es) &&
                    rows_aligned(y, y_stride, 0, es, kV * es);
  const bool wide_state = rows_aligned(state, dim, 0, es, kV * es);
  CR_MODEL_TYPE(dt, CR_CONV_WIDTH(width, {
    CR_LAUNCH(kKCausalConvStep, s,
              causal_conv_step_kernel<T, K><<<(unsigned)(batch * col_blocks), kConvThreads, 0, s>>>(
                  static_cast<const T*>(x), x_stride, static_cast<T*>(state), state_rows, slots,
                  index_bytes, weight, bias, activation == CR_ACT_SILU, dim, col_blocks, wide,
                  wide_state, static_cast<T*>(y), y_stride));
  }));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
