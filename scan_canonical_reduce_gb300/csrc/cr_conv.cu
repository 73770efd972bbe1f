// Depthwise causal convolution over time, its gradient, and its single-token
// form.
//
//   pre[t] = bias + sum_{k<K} w[k] x[t-(K-1)+k],   y[t] = act(pre[t])
//   dpre[t] = dy[t] act'(pre[t])
//   dx[p] = sum_{k<K} w[k] dpre[p+(K-1)-k],  dw[k] = sum_t dpre[t] x[t-(K-1)+k]
//
// A thread takes four neighbouring channels, as two pairs for the packed
// arithmetic, and a run of time steps, and keeps the last K inputs (backward:
// and the last K of dpre) in registers, so that each input is read once, plus
// K-1 steps of halo a run. Steps go in groups, the next group's reads in
// flight.
//
// Measured, bf16, 4 x 4096 steps of 4096 channels, K = 4, SiLU: forward 60 us
// (268 MB, 4.4 TB/s), backward 105 us (403 MB, 3.8 TB/s) and 10 us for the sums
// over runs; DRAM and issue bound both (about 45 and 80 instructions for a step
// of four channels). One token of 64 streams of 4096 channels 5 us with its
// call, 3.1 us of it on the device.
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

constexpr int kConvThreads = 128;
constexpr int kV = 4;  // channels a thread

// Where a thread's four channels are. Wide: neighbours, accessed at once.
// Otherwise (rows that start anywhere) 32 apart, so that a warp's accesses,
// one channel a thread, are consecutive.
template <bool kWide>
struct Channels {
  static constexpr int kStep = kWide ? 1 : 32;
  // block: of kConvThreads kV channels
  static __device__ __forceinline__ int64_t first(int64_t block) {
    if (kWide) return (block * kConvThreads + threadIdx.x) * kV;
    return block * kConvThreads * kV + threadIdx.x / 32 * 32 * kV + threadIdx.x % 32;
  }
  static __device__ __forceinline__ int have(int64_t c, int64_t dim) {
    const int64_t n = (dim - c + kStep - 1) / kStep;
    return (int)min((int64_t)kV, n);
  }
};

template <class T, bool kWide>
using Four = Raw<T, kV, kWide, Channels<kWide>::kStep>;

template <class T, bool kWide>
__device__ __forceinline__ void read_four(const T* p, bool whole, int have, float (&f)[kV]) {
  Four<T, kWide> r;
  r.load(p, whole, have);
#pragma unroll
  for (int j = 0; j < kV; ++j) f[j] = r.get(j);
}

template <class T, bool kWide>
__device__ __forceinline__ void write_four(T* p, bool whole, int have, const float (&f)[kV]) {
  store_raw<T, kV, kWide, Channels<kWide>::kStep>(p, whole, have, f);
}

struct ConvShape {
  int64_t batch, len, dim;
  int64_t run;        // steps a thread takes
  int64_t runs;       // of a sequence (at least 1)
  int64_t col_blocks; // blocks along the channels
};

// Runs of 64 steps read 5 % of halo (K = 4) and keep the backward's partial
// sums small; where that leaves too few threads they are halved, down to 16.
// A rule on sizes alone: the sums over time depend on it.
ConvShape conv_shape(int64_t batch, int64_t len, int64_t dim) {
  ConvShape c;
  c.batch = batch;
  c.len = len;
  c.dim = dim;
  c.run = 64;
  while (c.run > 16 && batch * ceil_div(len, c.run) * ceil_div(dim, kV) < 100000) c.run /= 2;
  c.runs = len > 0 ? ceil_div(len, c.run) : 1;
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
  bool silu, wide, wide_state, wide_weight;
};

// Input at extended time t (t < 0: the state's) of channels c .. c + have.
template <class T, int K, bool kWide>
__device__ __forceinline__ void conv_input(const ConvIn<T>& in, const ConvShape& sh, int64_t b,
                                           int64_t t, int64_t c, int have, float (&f)[kV]) {
  if (t >= 0) {
    read_four<T, kWide>(in.x + b * in.bs + t * in.ts + c, in.wide && have == kV, have, f);
  } else if (in.state != nullptr) {
    read_four<T, kWide>(in.state + (b * (K - 1) + (K - 1 + t)) * sh.dim + c,
                        in.wide_state && have == kV, have, f);
  } else {
#pragma unroll
    for (int j = 0; j < kV; ++j) f[j] = 0.0f;
  }
}

// Four channels as two pairs.
struct Quad {
  F2 p[2];
};

__device__ __forceinline__ Quad quad_of(const float (&f)[kV]) {
  return {{pack2(f[0], f[1]), pack2(f[2], f[3])}};
}
__device__ __forceinline__ void unquad(const Quad& q, float (&f)[kV]) {
  unpack2(q.p[0], f[0], f[1]);
  unpack2(q.p[1], f[2], f[3]);
}
template <class R>
__device__ __forceinline__ Quad quad(const R& r) {
  return {{pack2(r.get(0), r.get(1)), pack2(r.get(2), r.get(3))}};
}

template <int K, bool kWide>
__device__ __forceinline__ void conv_weights(const float* weight, const float* bias,
                                             bool wide_weight, int64_t c, int have, Quad (&w)[K],
                                             Quad& b0) {
  constexpr int kStep = Channels<kWide>::kStep;
  float f[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) f[j] = (bias != nullptr && j < have) ? bias[c + j * kStep] : 0.0f;
  b0 = quad_of(f);
  float v[K][kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const float* q = weight + (c + j * kStep) * K;
    if (K != 3 && wide_weight && j < have) {  // a channel's taps at once
      Raw<float, K == 3 ? 1 : K> r;
      r.load(q, true, K);
#pragma unroll
      for (int k = 0; k < K; ++k) v[k][j] = r.get(K == 3 ? 0 : k);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k][j] = j < have ? q[k] : 0.0f;
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = quad_of(v[k]);
}

// pre = bias + sum_k w[k] x[k], k upwards.
template <int K>
__device__ __forceinline__ Quad conv_pre(const Quad (&w)[K], const Quad& b0, const Quad* x) {
  Quad p = b0;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) p.p[i] = fma2(w[k].p[i], x[k].p[i], p.p[i]);
  return p;
}

__device__ __forceinline__ void conv_act(bool silu, float (&f)[kV]) {
  if (silu) {
#pragma unroll
    for (int j = 0; j < kV; ++j) f[j] = f[j] * sigmoid(f[j]);
  }
}

// U rows of a tensor's four channels from p on. kFull: all of them exist and
// are read whole; otherwise the first `rows` do, the others are zero and not
// read. Most groups are full, and the checks cost more than their arithmetic.
template <bool kFull, class T, int U, class R>
__device__ __forceinline__ void load_group(const T* p, int64_t ts, int rows, bool wide, int have,
                                           R (&r)[U]) {
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (kFull) r[i].load(p + i * ts, true, kV);
    else if (i < rows) r[i].load(p + i * ts, wide, have);
    else r[i].zero();
  }
}

template <bool kFull, bool kWide, class T>
__device__ __forceinline__ void store_row(T* p, bool wide, int have, const float (&f)[kV]) {
  write_four<T, kWide>(p, kFull || wide, kFull ? kV : have, f);
}

#ifndef CR_CONV_FORWARD
#define CR_CONV_FORWARD 8
#endif
constexpr int kForward = CR_CONV_FORWARD, kBackward = 4;  // steps of a group

// Blocks an SM (registers): forward 4 (128 registers; 5: the same, 6: 74 us),
// backward 3 (159 registers, 108 us; 4: 115, 5: 208, with spills).
#ifndef CR_CONV_BLOCKS
#define CR_CONV_BLOCKS 4
#endif
#ifndef CR_CONV_BACK_BLOCKS
#define CR_CONV_BACK_BLOCKS 3
#endif
template <class T, int K, bool kWide>
__global__ void __launch_bounds__(kConvThreads, CR_CONV_BLOCKS)
causal_conv_kernel(ConvIn<T> in, ConvShape sh, T* __restrict__ y, int64_t ybs, int64_t yts,
                   bool wide_y, T* __restrict__ final_state) {
  constexpr int U = kForward;
  int64_t c, run;
  const int64_t b = divide(divide(blockIdx.x, sh.col_blocks, c), sh.runs, run);
  c = Channels<kWide>::first(c);
  if (c >= sh.dim) return;
  const int have = Channels<kWide>::have(c, sh.dim);
  const int64_t len = sequence_length(in.lengths, in.index_bytes, b, sh.len);
  const int64_t t0 = run * sh.run, t1 = min(sh.len, t0 + sh.run), stop = min(t1, len);
  const bool wy = wide_y && have == kV, wx = in.wide && have == kV;
  y += b * ybs + c;

  if (t0 < stop) {
    const int rows = (int)(stop - t0);
    const T* x = in.x + b * in.bs + t0 * in.ts + c;  // of the next group
    T* o = y + t0 * yts;
    Four<T, kWide> next[U];
    load_group<false, T, U>(x, in.ts, rows, wx, have, next);
    x += U * in.ts;
    Quad w[K], b0, win[K - 1 + U];
    conv_weights<K, kWide>(in.weight, in.bias, in.wide_weight, c, have, w, b0);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      float f[kV];
      conv_input<T, K, kWide>(in, sh, b, t0 - (K - 1) + k, c, have, f);
      win[k] = quad_of(f);
    }
    auto group = [&](auto full, int left) {
      constexpr bool kFull = decltype(full)::value;
#pragma unroll
      for (int u = 0; u < U; ++u) win[K - 1 + u] = quad(next[u]);
      load_group<kFull, T, U>(x, in.ts, left - U, wx, have, next);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[kV];
        unquad(conv_pre<K>(w, b0, win + u), f);
        conv_act(in.silu, f);
        if (kFull || u < left) store_row<kFull, kWide>(o + u * yts, wy, have, f);
      }
#pragma unroll
      for (int k = 0; k < K - 1; ++k) win[k] = win[U + k];
      x += U * in.ts;
      o += U * yts;
    };
    int left = rows;
    if (kWide ? wx && wy : have == kV) {
#pragma unroll 1
      for (; left >= 2 * U; left -= U) group(std::true_type{}, left);
    }
#pragma unroll 1
    for (; left > 0; left -= U) group(std::false_type{}, left);
  }
  const float zero[kV] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t t = max(t0, len); t < t1; ++t) write_four<T, kWide>(y + t * yts, wy, have, zero);
  if (run == 0 && final_state != nullptr) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      float f[kV];
      conv_input<T, K, kWide>(in, sh, b, len - (K - 1) + j, c, have, f);
      write_four<T, kWide>(final_state + (b * (K - 1) + j) * sh.dim + c,
                           in.wide_state && have == kV, have, f);
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
template <class T, int K, bool kWide>
__global__ void __launch_bounds__(kConvThreads, CR_CONV_BACK_BLOCKS)
causal_conv_backward_kernel(ConvIn<T> in, ConvShape sh, ConvBack<T> g) {
  constexpr int U = kBackward;
  int64_t c, run;
  const int64_t b = divide(divide(blockIdx.x, sh.col_blocks, c), sh.runs, run);
  c = Channels<kWide>::first(c);
  if (c >= sh.dim) return;
  const int have = Channels<kWide>::have(c, sh.dim);
  const int64_t len = sequence_length(in.lengths, in.index_bytes, b, sh.len);
  const int64_t t0 = run * sh.run, t1 = min(sh.len, t0 + sh.run);
  const bool wide = in.wide && have == kV, wide_dx = g.wide_dx && have == kV;
  const bool wide_state = in.wide_state && have == kV;
  T* dx = g.dx + b * g.dxbs + c;
  const int64_t final0 = len - (K - 1);  // the first of the state's positions

  Quad dw[K], db = {{0, 0}};
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k] = {{0, 0}};
  if (t0 < len || run == 0) {
    const T* x = in.x + b * in.bs + t0 * in.ts + c;  // of the next group
    const T* dy = g.dy + b * g.dybs + t0 * g.dyts + c;
    Four<T, kWide> nx[U], ny[U];
    const int rows = (int)min(len - t0, (int64_t)1 << 30);  // that exist, from t0 on
    load_group<false, T, U>(x, in.ts, rows, wide, have, nx);
    load_group<false, T, U>(dy, g.dyts, rows, wide, have, ny);
    x += U * in.ts;
    dy += U * g.dyts;
    Quad w[K], b0, win[K - 1 + U], dp[K - 1 + U];
    conv_weights<K, kWide>(in.weight, in.bias, in.wide_weight, c, have, w, b0);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      float f[kV];
      conv_input<T, K, kWide>(in, sh, b, t0 - (K - 1) + k, c, have, f);
      win[k] = quad_of(f);
      dp[k] = {{0, 0}};
    }
    const int own = (int)(t1 - t0);  // steps of this run
    // Steps past the sequence add nothing, even where dy's zeros would meet a
    // NaN or an infinity in the window.
    const int live = min(own, rows);
    T* o = dx + (t0 - (K - 1)) * g.dxts;  // of position t - (K - 1)
    // After step t the window of dpre ends at t, which completes dx at t -
    // (K - 1). Full: steps and positions all lie inside the run and the
    // sequence (and the next group's rows inside the sequence).
    auto group = [&](auto full, int s) {
      constexpr bool kFull = decltype(full)::value;
      Quad d[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        win[K - 1 + u] = quad(nx[u]);
        d[u] = quad(ny[u]);
      }
      load_group<kFull, T, U>(x, in.ts, rows - s - U, wide, have, nx);
      load_group<kFull, T, U>(dy, g.dyts, rows - s - U, wide, have, ny);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (in.silu) {
          float f[kV], sg[kV];
          unquad(conv_pre<K>(w, b0, win + u), f);
#pragma unroll
          for (int j = 0; j < kV; ++j) sg[j] = sigmoid(f[j]);
          // act' = s (1 + pre (1 - s)) = s + (pre s) (1 - s)
#pragma unroll
          for (int j = 0; j < kV; ++j) f[j] = fmaf(f[j] * sg[j], 1.0f - sg[j], sg[j]);
          const Quad a = quad_of(f);
#pragma unroll
          for (int j = 0; j < 2; ++j) d[u].p[j] = mul2(d[u].p[j], a.p[j]);
        }
        if (!kFull && s + u >= rows) d[u] = {{0, 0}};
        dp[K - 1 + u] = d[u];
        if (kFull || s + u < live) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            db.p[j] = add2_products(db.p[j], d[u].p[j]);
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k].p[j] = fma2(d[u].p[j], win[u + k].p[j], dw[k].p[j]);
          }
        }
        const int q = s + u - (K - 1);  // the position, from t0
        if (kFull || ((q >= 0 || run == 0) && q < own)) {  // others: the run before's
          Quad v = {{0, 0}};
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              v.p[j] = fma2(w[k].p[j], dp[u + K - 1 - k].p[j], v.p[j]);
          float f[kV];
          unquad(v, f);
          if (kFull) {
            store_row<true, kWide>(o + u * g.dxts, wide_dx, have, f);
          } else {
            const int64_t p = t0 + q;
            if (g.dfinal != nullptr && p >= final0 && p < len) {
              float e[kV];
              read_four<T, kWide>(g.dfinal + (b * (K - 1) + (p - final0)) * sh.dim + c, wide_state,
                                  have, e);
#pragma unroll
              for (int j = 0; j < kV; ++j) f[j] += e[j];
            }
            if (p >= 0) {
              if (g.dx != nullptr) store_row<false, kWide>(o + u * g.dxts, wide_dx, have, f);
            } else if (g.dstate != nullptr) {
              write_four<T, kWide>(g.dstate + (b * (K - 1) + (K - 1 + p)) * sh.dim + c, wide_state,
                                   have, f);
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < K - 1; ++k) {
        win[k] = win[U + k];
        dp[k] = dp[U + k];
      }
      x += U * in.ts;
      dy += U * g.dyts;
      o += U * g.dxts;
    };
    static_assert(U >= K - 1, "the group after the first has no position before the run");
    int s = 0;
    group(std::false_type{}, s);
    s += U;
    if ((kWide ? wide && wide_dx : have == kV) && g.dx != nullptr) {
      const int full = (int)min((int64_t)own, (int64_t)rows - U);  // the last with a next group
#pragma unroll 1
      for (; s + U <= full; s += U) group(std::true_type{}, s);
    }
#pragma unroll 1
    for (; s < own + K - 1; s += U) group(std::false_type{}, s);
  } else if (g.dx != nullptr) {
    const float zero[kV] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t t = t0; t < t1; ++t) write_four<T, kWide>(dx + t * g.dxts, wide_dx, have, zero);
  }
  // [run][K + 1][dim]: neighbouring threads write neighbours
  float* part = g.part + (b * sh.runs + run) * (K + 1) * sh.dim + c;
  const bool wp = kWide && sh.dim % kV == 0;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    float f[kV];
    unquad(k < K ? dw[k < K ? k : 0] : db, f);
    write_four<float, kWide>(part + k * sh.dim, wp, have, f);
  }
}

// Sums the runs' partials: eight threads take every eighth run of a column
// (tap and channel) in order, then one adds the eight.
__global__ void __launch_bounds__(256)
causal_conv_sum_kernel(const float* __restrict__ part, int64_t parts, int64_t dim, int K,
                       float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float sums[8][32];
  const int64_t n = dim * (K + 1);
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < n) {
#pragma unroll 8
    for (int64_t p = row; p < parts; p += 8) s += part[p * n + i];
  }
  sums[row][lane] = s;
  __syncthreads();
  if (row != 0 || i >= n) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) s += sums[r][lane];
  int64_t d;
  const int k = (int)divide(i, dim, d);
  if (k < K) dweight[d * K + k] = s;
  else if (dbias != nullptr) dbias[d] = s;
}

template <class T, int K, bool kWide>
__global__ void __launch_bounds__(kConvThreads)
causal_conv_step_kernel(const T* __restrict__ x, int64_t x_stride, T* __restrict__ state,
                        int64_t state_rows, const void* __restrict__ slots, int index_bytes,
                        const float* __restrict__ weight, const float* __restrict__ bias,
                        bool silu, int64_t dim, int64_t col_blocks, bool wide, bool wide_state,
                        bool wide_weight,
                        T* __restrict__ y, int64_t y_stride) {
  int64_t c;
  const int64_t b = divide(blockIdx.x, col_blocks, c);
  c = Channels<kWide>::first(c);
  if (c >= dim) return;
  const int have = Channels<kWide>::have(c, dim);
  const bool full = have == kV;
  const int64_t row = slots != nullptr ? load_index(slots, index_bytes, b) : b;
  float o[kV] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (row >= 0 && row < state_rows) {
    Quad win[K];
    T* st = state + row * (K - 1) * dim + c;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      float f[kV];
      read_own<T, kV, kWide, Channels<kWide>::kStep>(st + k * dim, wide_state && full, have, f);
      win[k] = quad_of(f);
    }
    Quad w[K], b0;
    conv_weights<K, kWide>(weight, bias, wide_weight, c, have, w, b0);
    float f[kV];
    read_four<T, kWide>(x + b * x_stride + c, wide && full, have, f);
    win[K - 1] = quad_of(f);
    unquad(conv_pre<K>(w, b0, win), o);
    conv_act(silu, o);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      unquad(win[k + 1], f);
      write_four<T, kWide>(st + k * dim, wide_state && full, have, f);
    }
  }
  write_four<T, kWide>(y + b * y_stride + c, wide && full, have, o);
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
  in.wide_weight = ptr_aligned(a->weight, (size_t)a->width * 4);
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
  if (a->len > 0 && (y == nullptr || (a->len > 1 && y_time_stride < a->dim) ||
                     (a->batch > 1 && y_batch_stride < a->dim)))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(y, es) || !ptr_aligned(final_state, es) ||
      overwrites({y, final_state}, {a->x, a->weight, a->bias, a->state, a->lengths}))
    return CR_ERR_INVALID_ARG;
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
              (wide && wide_y ? causal_conv_kernel<T, K, true> : causal_conv_kernel<T, K, false>)
              <<<blocks, kConvThreads, 0, s>>>(
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
  return round256((size_t)(batch * sh.runs) * (size_t)dim * (width + 1) * 4) + kStatusBytes;
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
    if (g->dy == nullptr) return CR_ERR_INVALID_ARG;
    if (g->dx != nullptr && ((a->len > 1 && g->dx_time_stride < a->dim) ||
                             (a->batch > 1 && g->dx_batch_stride < a->dim)))
      return CR_ERR_INVALID_ARG;
  }
  if (!ptr_aligned(g->dy, es) || !ptr_aligned(g->dx, es) || !ptr_aligned(g->dfinal, es) ||
      !ptr_aligned(g->dstate, es) || !ptr_aligned(g->dweight, 4) || !ptr_aligned(g->dbias, 4) ||
      overwrites({g->dx, g->dweight, g->dbias, g->dstate},
                 {a->x, a->weight, a->bias, a->state, a->lengths, g->dy, g->dfinal}))
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
      gb.part = reinterpret_cast<float*>(past_status(ws));
      gb.wide_dx = wide_dx;
      CR_LAUNCH(kKCausalConvBackward, s,
                (wide && wide_dx ? causal_conv_backward_kernel<T, K, true>
                                 : causal_conv_backward_kernel<T, K, false>)
                <<<blocks, kConvThreads, 0, s>>>(
                    conv_in<T>(a, wide, wide_state), sh, gb));
    }));
    if (cudaGetLastError() != cudaSuccess) return CR_ERR_CUDA;
  }
  const int64_t n = a->dim * (a->width + 1);
  CR_LAUNCH(kKCausalConvSum, s,
            causal_conv_sum_kernel<<<(unsigned)ceil_div(n, 32), 256, 0, s>>>(
                reinterpret_cast<const float*>(past_status(ws)), a->batch * sh.runs, a->dim, a->width, g->dweight,
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
  if (x == nullptr || weight == nullptr || y == nullptr ||
      overwrites({y}, {x, state, slots, weight, bias}) ||
      overwrites({state}, {x, slots, weight, bias}) ||
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
              (wide && wide_state ? causal_conv_step_kernel<T, K, true>
                                  : causal_conv_step_kernel<T, K, false>)
              <<<(unsigned)(batch * col_blocks), kConvThreads, 0, s>>>(
                  static_cast<const T*>(x), x_stride, static_cast<T*>(state), state_rows, slots,
                  index_bytes, weight, bias, activation == CR_ACT_SILU, dim, col_blocks, wide,
                  wide_state, ptr_aligned(weight, (size_t)width * 4), static_cast<T*>(y),
                  y_stride));
  }));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
