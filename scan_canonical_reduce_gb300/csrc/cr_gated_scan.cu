// Gated linear recurrence over time, its gradient, and its single-token form.
//
//   a[t] = sigmoid(gate[t]), r[t] = 1 - a[t] = sigmoid(-gate[t])
//   h[t] = a[t] h[t-1] + r[t] x[t],   y[t] = h[t] silu(z[t])
//   G[t] = dy[t] silu(z[t]) + a[t+1] G[t+1]
//   dx = r G,  dgate = (h[t-1] - x) G a r,  dz = dy h silu'(z)
//
// What is kept of a gate is the smaller of a and r, with the gate's sign. Where
// a memory is long, a is near 1 and has few digits of r left: a step that
// multiplied by it would forget at a rate that is off by 2^-25 / r. So
//   gate >= 0:  h + r (x - h),  a G = G - r G
//   gate < 0:   x + a (h - x),  a G = a G.
#include <algorithm>
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

constexpr int kGateCheckpoint = 16;

template <class T>
struct Strided {
  const T* p;
  int64_t bs, ts;
};

template <class T>
struct GateIn {
  int64_t batch, len, dim;
  Strided<T> x, gate, z;
  const float* state;
  const void* lengths;
  int32_t index_bytes;
};

// The smaller of a and r, negative where that is a.
__device__ __forceinline__ float gate_coef(float g) {
  const float e = exp2_fast(fabsf(g) * -kLog2e);
  return copysignf(e * reciprocal(1.0f + e), g);
}
__device__ __forceinline__ bool holds(float c) { return __float_as_int(c) >= 0; }
__device__ __forceinline__ float gate_step(float c, float h, float x) {
  return fmaf(c, x - h, holds(c) ? h : x);
}
__device__ __forceinline__ float take(float c) { return holds(c) ? c : 1.0f + c; }  // r
__device__ __forceinline__ float forget(float c, float G) {  // a G
  return holds(c) ? fmaf(-c, G, G) : -c * G;
}

template <class T>
__global__ void __launch_bounds__(128)
gated_scan_kernel(GateIn<T> in, T* __restrict__ y, int64_t ybs, int64_t yts, float* final_state,
                  float* __restrict__ checkpoints, int64_t n_check) {
  const int64_t per = (in.dim + 127) / 128;
  int64_t blk;
  const int64_t b = divide(blockIdx.x, per, blk), d = blk * 128 + threadIdx.x;
  if (d >= in.dim) return;
  const int64_t n = sequence_length(in.lengths, in.index_bytes, b, in.len);
  float h = in.state != nullptr ? in.state[b * in.dim + d] : 0.0f;
  for (int64_t t = 0; t < n; ++t) {
    if (checkpoints != nullptr && t % kGateCheckpoint == 0)
      checkpoints[(b * n_check + t / kGateCheckpoint) * in.dim + d] = h;
    const float x = to_f32(in.x.p[b * in.x.bs + t * in.x.ts + d]);
    h = gate_step(gate_coef(to_f32(in.gate.p[b * in.gate.bs + t * in.gate.ts + d])), h, x);
    float o = h;
    if (in.z.p != nullptr) {
      const float z = to_f32(in.z.p[b * in.z.bs + t * in.z.ts + d]);
      o *= z * sigmoid(z);
    }
    y[b * ybs + t * yts + d] = from_f32<T>(o);
  }
  for (int64_t t = n; t < in.len; ++t) y[b * ybs + t * yts + d] = from_f32<T>(0.0f);
  if (final_state != nullptr) final_state[b * in.dim + d] = h;
}

template <class T>
struct GateOut {
  T *dx, *dgate, *dz;  // contiguous
  float* dstate;
};

template <class T>
__global__ void __launch_bounds__(128)
gated_scan_backward_kernel(GateIn<T> in, Strided<T> dy, const float* __restrict__ dfinal,
                           const float* __restrict__ checkpoints, int64_t n_check, GateOut<T> out) {
  const int64_t per = (in.dim + 127) / 128;
  int64_t blk;
  const int64_t b = divide(blockIdx.x, per, blk), d = blk * 128 + threadIdx.x;
  if (d >= in.dim) return;
  const int64_t n = sequence_length(in.lengths, in.index_bytes, b, in.len);
  for (int64_t t = n; t < in.len; ++t) {
    const int64_t at = (b * in.len + t) * in.dim + d;
    out.dx[at] = out.dgate[at] = from_f32<T>(0.0f);
    if (in.z.p != nullptr) out.dz[at] = from_f32<T>(0.0f);
  }
  float G = dfinal != nullptr ? dfinal[b * in.dim + d] : 0.0f;
  for (int64_t t1 = (n + kGateCheckpoint - 1) / kGateCheckpoint; t1 > 0; --t1) {
    const int64_t t0 = (t1 - 1) * kGateCheckpoint;
    const int m = (int)min((int64_t)kGateCheckpoint, n - t0);
    float before[kGateCheckpoint];
    float h = checkpoints[(b * n_check + t1 - 1) * in.dim + d];
    for (int k = 0; k < m; ++k) {
      before[k] = h;
      const float x = to_f32(in.x.p[b * in.x.bs + (t0 + k) * in.x.ts + d]);
      h = gate_step(gate_coef(to_f32(in.gate.p[b * in.gate.bs + (t0 + k) * in.gate.ts + d])), h,
                    x);
    }
    for (int k = m - 1; k >= 0; --k) {
      const int64_t t = t0 + k, at = (b * in.len + t) * in.dim + d;
      const float x = to_f32(in.x.p[b * in.x.bs + t * in.x.ts + d]);
      const float c = gate_coef(to_f32(in.gate.p[b * in.gate.bs + t * in.gate.ts + d]));
      float g = to_f32(dy.p[b * dy.bs + t * dy.ts + d]);
      if (in.z.p != nullptr) {
        const float z = to_f32(in.z.p[b * in.z.bs + t * in.z.ts + d]), s = sigmoid(z);
        out.dz[at] = from_f32<T>(g * h * (s * (1.0f + z * (1.0f - s))));
        g *= z * s;
      }
      G = G + g;
      out.dx[at] = from_f32<T>(take(c) * G);
      out.dgate[at] = from_f32<T>((before[k] - x) * G * (fabsf(c) * (1.0f - fabsf(c))));
      G = forget(c, G);
      h = before[k];
    }
  }
  if (out.dstate != nullptr) out.dstate[b * in.dim + d] = G;
}

template <class T>
__global__ void __launch_bounds__(128)
gated_scan_step_kernel(GateIn<T> in, float* __restrict__ state, int64_t rows, const void* slots,
                       T* __restrict__ y, int64_t ybs) {
  const int64_t d = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (d >= in.dim) return;
  for (int64_t b = blockIdx.y; b < in.batch; b += gridDim.y) {
    const int64_t row = slots != nullptr ? load_index(slots, in.index_bytes, b) : b;
    float o = 0.0f;
    if (row >= 0 && row < rows) {
      float h = state[row * in.dim + d];
      const float x = to_f32(in.x.p[b * in.x.bs + d]);
      h = gate_step(gate_coef(to_f32(in.gate.p[b * in.gate.bs + d])), h, x);
      state[row * in.dim + d] = h;
      o = h;
      if (in.z.p != nullptr) {
        const float z = to_f32(in.z.p[b * in.z.bs + d]);
        o *= z * sigmoid(z);
      }
    }
    y[b * ybs + d] = from_f32<T>(o);
  }
}

template <class T>
GateIn<T> gate_in(const cr_gated_scan_args* a) {
  return {a->batch, a->len, a->dim,
          {static_cast<const T*>(a->x), a->x_batch_stride, a->x_time_stride},
          {static_cast<const T*>(a->gate), a->gate_batch_stride, a->gate_time_stride},
          {static_cast<const T*>(a->z), a->z_batch_stride, a->z_time_stride},
          a->state, a->lengths, a->index_bytes};
}

cr_status check_gate(const cr_gated_scan_args* a, bool step) {
  if (a == nullptr) return CR_ERR_INVALID_ARG;
  const size_t es = model_esize(a->dt);
  if (es == 0 || a->batch < 0 || a->len < 0 || a->dim < 0 || (step && a->len != 1))
    return CR_ERR_INVALID_ARG;
  for (int64_t v : {a->x_batch_stride, a->x_time_stride, a->gate_batch_stride,
                    a->gate_time_stride, a->z_batch_stride, a->z_time_stride})
    if (v < 0) return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->len > 0 && a->dim > 0 && (a->x == nullptr || a->gate == nullptr))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(a->x, es) || !ptr_aligned(a->gate, es) || !ptr_aligned(a->z, es))
    return CR_ERR_INVALID_ARG;
  if (!step && (!ptr_aligned(a->state, 4) ||
                (a->lengths != nullptr && (!index_width_ok(a->index_bytes) ||
                                           !ptr_aligned(a->lengths, a->index_bytes)))))
    return CR_ERR_INVALID_ARG;
  return CR_OK;
}

}  // namespace
}  // namespace cr

extern "C" {

int64_t cr_gated_scan_checkpoints(int64_t len) {
  return len <= 0 ? 0 : cr::ceil_div(len, cr::kGateCheckpoint);
}

cr_status cr_gated_scan(const cr_gated_scan_args* a, void* y, int64_t y_batch_stride,
                        int64_t y_time_stride, float* final_state, float* checkpoints,
                        void* stream) {
  using namespace cr;
  const cr_status ok = check_gate(a, false);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt);
  if (y_batch_stride < 0 || y_time_stride < 0 || !ptr_aligned(y, es) ||
      !ptr_aligned(final_state, 4) || !ptr_aligned(checkpoints, 4))
    return CR_ERR_INVALID_ARG;
  if (a->batch == 0 || a->dim == 0) return CR_OK;
  if (a->len > 0 && (y == nullptr || (a->len > 1 && y_time_stride < a->dim) ||
                     (a->batch > 1 && y_batch_stride < a->dim)))
    return CR_ERR_INVALID_ARG;
  if (overwrites({y, final_state, checkpoints}, {a->x, a->gate, a->z, a->lengths}) ||
      overwrites({y, checkpoints}, {a->state}))
    return CR_ERR_INVALID_ARG;
  if (a->len == 0 && final_state == nullptr) return CR_OK;
  const int64_t per = ceil_div(a->dim, 128);
  if (a->batch > kMaxBlocks / per) return CR_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    CR_LAUNCH(kKGatedScan, s,
              gated_scan_kernel<T><<<(unsigned)(a->batch * per), 128, 0, s>>>(
                  gate_in<T>(a), static_cast<T*>(y), y_batch_stride, y_time_stride, final_state,
                  checkpoints, cr_gated_scan_checkpoints(a->len)));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

cr_status cr_gated_scan_backward(const cr_gated_scan_args* a, const cr_gated_scan_grads* g,
                                 void* stream) {
  using namespace cr;
  const cr_status ok = check_gate(a, false);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt);
  if (g == nullptr || g->dy_batch_stride < 0 || g->dy_time_stride < 0) return CR_ERR_INVALID_ARG;
  for (const void* p : {g->dy, (const void*)g->dx, (const void*)g->dgate, (const void*)g->dz})
    if (!ptr_aligned(p, es)) return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(g->dfinal, 4) || !ptr_aligned(g->checkpoints, 4) || !ptr_aligned(g->dstate, 4))
    return CR_ERR_INVALID_ARG;
  if (a->batch == 0 || a->dim == 0) return CR_OK;
  if (a->len > 0 && (g->dy == nullptr || g->checkpoints == nullptr || g->dx == nullptr ||
                     g->dgate == nullptr || (a->z != nullptr && g->dz == nullptr)))
    return CR_ERR_INVALID_ARG;
  if (overwrites({g->dx, g->dgate, g->dz, g->dstate},
                 {a->x, a->gate, a->z, a->state, a->lengths, g->dy, g->dfinal, g->checkpoints}))
    return CR_ERR_INVALID_ARG;
  if (a->len == 0 && g->dstate == nullptr) return CR_OK;
  const int64_t per = ceil_div(a->dim, 128);
  if (a->batch > kMaxBlocks / per) return CR_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    const Strided<T> dy = {static_cast<const T*>(g->dy), g->dy_batch_stride, g->dy_time_stride};
    const GateOut<T> out = {static_cast<T*>(g->dx), static_cast<T*>(g->dgate),
                            static_cast<T*>(g->dz), g->dstate};
    CR_LAUNCH(kKGatedScanBackward, s,
              gated_scan_backward_kernel<T><<<(unsigned)(a->batch * per), 128, 0, s>>>(
                  gate_in<T>(a), dy, g->dfinal, g->checkpoints,
                  cr_gated_scan_checkpoints(a->len), out));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

cr_status cr_gated_scan_step(const cr_gated_scan_args* a, float* state, int64_t state_rows,
                             const void* slots, void* y, int64_t y_batch_stride, void* stream) {
  using namespace cr;
  const cr_status ok = check_gate(a, true);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt);
  if (state_rows < 0 || y_batch_stride < 0) return CR_ERR_INVALID_ARG;
  if (slots != nullptr ? !index_width_ok(a->index_bytes) || !ptr_aligned(slots, a->index_bytes)
                       : state_rows < a->batch)
    return CR_ERR_INVALID_ARG;
  if (a->batch == 0 || a->dim == 0) return CR_OK;
  if (y == nullptr || (state == nullptr && state_rows > 0) ||
      (a->batch > 1 && y_batch_stride < a->dim) || y == (void*)state ||
      overwrites({y, state}, {a->x, a->gate, a->z, slots}))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(y, es) || !ptr_aligned(state, 4)) return CR_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t blocks = ceil_div(a->dim, 128);
  if (blocks > kMaxBlocks) return CR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks, (unsigned)std::min<int64_t>(a->batch, 65535));
  CR_MODEL_TYPE(a->dt, {
    CR_LAUNCH(kKGatedScanStep, s,
              gated_scan_step_kernel<T><<<grid, 128, 0, s>>>(gate_in<T>(a), state, state_rows,
                                                            slots, static_cast<T*>(y),
                                                            y_batch_stride));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
