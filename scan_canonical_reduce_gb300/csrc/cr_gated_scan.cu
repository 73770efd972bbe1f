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

#include <cooperative_groups.h>

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
__device__ __forceinline__ float keep(float c) { return (holds(c) ? 1.0f : 0.0f) - c; }  // a
__device__ __forceinline__ float take(float c) { return holds(c) ? c : 1.0f + c; }  // r
__device__ __forceinline__ float forget(float c, float G) {  // a G
  return holds(c) ? fmaf(-c, G, G) : -c * G;
}

// What a run of steps does to the state: h -> L + P h. Where P is near 1 its
// digits are in Q = 1 - P, where it is near 0 in P: kept is Q, or -P from 1 -
// 2^-7 on (below that, P's error is 2^-17 of itself at most).
__device__ __forceinline__ float map_keep(float Q, float P) {
  return Q <= 1.0f - 0x1p-7f ? Q : -P;
}
__device__ __forceinline__ float map_apply(float L, float F, float h) {
  const float v = fmaf(-F, h, L);
  return __float_as_int(F) >= 0 ? v + h : v;
}
// The map L, F after the map l, f: both as (L, F).
__device__ __forceinline__ void map_join(float& L, float& F, float l, float f) {
  const bool n0 = __float_as_int(F) >= 0, n1 = __float_as_int(f) >= 0;
  const float P0 = n0 ? 1.0f - F : -F, P1 = n1 ? 1.0f - f : -f;
  const float Q0 = n0 ? F : 1.0f + F, Q1 = n1 ? f : 1.0f + f;
  L = map_apply(l, f, L);
  F = map_keep(fmaf(Q1, P0, Q0), P0 * P1);
}

// A tile: 8 warps, each a run of kRun steps, a lane 32 bits of each step: one
// channel of binary32, two of 16 bits: neighbours (kWide), or 32 apart where
// rows start anywhere.
constexpr int kRun = kGateCheckpoint;
constexpr int kGateWarps = 8;
constexpr int kTileSteps = kRun * kGateWarps;
constexpr int kMostCluster = 16;

template <class T>
struct Lane {
  static constexpr int C = 4 / sizeof(T);  // channels
};

template <class T, bool kWide>
struct Word {
  static constexpr int C = Lane<T>::C;
  static __device__ __forceinline__ uint32_t load(const T* p, int have) {
    if constexpr (sizeof(T) == 4) {
      return have > 0 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
    } else if constexpr (kWide) {
      return have > 0 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
    } else {
      const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
      const uint32_t lo = have > 0 ? __ldg(q) : 0u, hi = have > 1 ? __ldg(q + 32) : 0u;
      return lo | hi << 16;
    }
  }
  static __device__ __forceinline__ float get(uint32_t w, int k) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(k ? w & 0xFFFF0000u : w << 16);
    else
      return __half2float(__ushort_as_half((unsigned short)(k ? w >> 16 : w & 0xFFFFu)));
  }
  static __device__ __forceinline__ void store(T* p, int have, const float (&f)[C]) {
    if constexpr (sizeof(T) == 4) {
      if (have > 0) *p = f[0];
    } else if constexpr (kWide) {
      if (have > 0) {
        Pack<T, 2> q;
        q.v[0] = from_f32<T>(f[0]);
        q.v[1] = from_f32<T>(f[1]);
        *reinterpret_cast<Pack<T, 2>*>(p) = q;
      }
    } else {
      if (have > 0) p[0] = from_f32<T>(f[0]);
      if (have > 1) p[32] = from_f32<T>(f[1]);
    }
  }
};

// Which channels a lane has.
template <class T, bool kWide>
struct Channels {
  static constexpr int C = Lane<T>::C;
  static constexpr int kStep = kWide ? 1 : 32;
  int64_t d;
  int have;
  __device__ Channels(int64_t group, int64_t dim) {
    const int lane = threadIdx.x % 32;
    d = group * 32 * C + (kWide ? lane * C : lane);
    have = d >= dim ? 0 : C == 1 || d + kStep >= dim ? 1 : 2;
    if (have == 0) d = 0;
  }
  __device__ __forceinline__ int64_t at(int k) const { return d + k * kStep; }
};

// The maps of a tile's warps and of a cluster's tiles, for this turn and the
// one before, which another block of the cluster may still be reading.
template <int C>
struct Joints {
  float2 warp[2][kGateWarps][32 * C];
  float2 tile[2][kMostCluster][32 * C];
};

// Gives the state that this warp's run starts from, and moves `carry` past all
// of the cluster's tiles. Run maps (L, F) are in time order for warps and
// blocks `first` to `last`.
template <int C, bool kBack>
__device__ __forceinline__ void join_runs(Joints<C>& j, int turn, int rank, int blocks,
                                          const float (&L)[C], const float (&F)[C],
                                          float (&carry)[C], float (&h)[C]) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int k = 0; k < C; ++k) j.warp[turn][warp][lane * C + k] = make_float2(L[k], F[k]);
  __syncthreads();
  // the tile's map, to every block of the cluster: warp w tells blocks w, w + 8
  if (warp < blocks) {
    float tl[C], tf[C];
#pragma unroll
    for (int i = 0; i < kGateWarps; ++i) {
      const int w = kBack ? kGateWarps - 1 - i : i;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const float2 m = j.warp[turn][w][lane * C + k];
        if (i == 0) tl[k] = m.x, tf[k] = m.y;
        else map_join(tl[k], tf[k], m.x, m.y);
      }
    }
    for (int to = warp; to < blocks; to += kGateWarps) {
      float2* p = cl.map_shared_rank(&j.tile[turn][rank][lane * C], to);
#pragma unroll
      for (int k = 0; k < C; ++k) p[k] = make_float2(tl[k], tf[k]);
    }
  }
  cl.sync();
#pragma unroll
  for (int k = 0; k < C; ++k) h[k] = carry[k];
  for (int i = 0; i < blocks; ++i) {
    const int r = kBack ? blocks - 1 - i : i;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const float2 m = j.tile[turn][r][lane * C + k];
      if (r == rank) h[k] = carry[k];
      carry[k] = map_apply(m.x, m.y, carry[k]);
    }
  }
#pragma unroll
  for (int i = 0; i < kGateWarps; ++i) {
    const int w = kBack ? kGateWarps - 1 - i : i;
    if (kBack ? w > warp : w < warp) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const float2 m = j.warp[turn][w][lane * C + k];
        h[k] = map_apply(m.x, m.y, h[k]);
      }
    }
  }
}

template <class T>
struct GateFwd {
  T* y;
  int64_t ybs, yts;
  float* final_state;
  float* checkpoints;
  int64_t n_check;
};

template <class T, bool kZ, bool kWide>
__global__ void __launch_bounds__(kGateWarps * 32, 2)
gated_scan_kernel(GateIn<T> in, GateFwd<T> out, int blocks) {
  constexpr int C = Lane<T>::C;
  using W = Word<T, kWide>;
  __shared__ Joints<C> joints;
  const int warp = threadIdx.x / 32;
  const int rank = (int)(blockIdx.x % (unsigned)blocks);
  const int64_t per = (in.dim + 32 * C - 1) / (32 * C);
  int64_t group;
  const int64_t b = divide(blockIdx.x / (unsigned)blocks, per, group);
  const Channels<T, kWide> ch(group, in.dim);
  const int64_t n = sequence_length(in.lengths, in.index_bytes, b, in.len);
  float carry[C];
#pragma unroll
  for (int k = 0; k < C; ++k)
    carry[k] = in.state != nullptr && k < ch.have ? in.state[b * in.dim + ch.at(k)] : 0.0f;
  const int64_t step = (int64_t)blocks * kTileSteps;
  int turn = 0;
  int64_t t0 = (int64_t)rank * kTileSteps + warp * kRun;  // this warp's run
  for (int64_t s0 = 0; s0 < n; s0 += step, t0 += step, turn ^= 1) {
    uint32_t x[kRun], z[kRun];
    float c[kRun][C];
    const int m = (int)max((int64_t)0, min((int64_t)kRun, n - t0));
    const T* px = in.x.p + b * in.x.bs + t0 * in.x.ts + ch.d;
    const T* pg = in.gate.p + b * in.gate.bs + t0 * in.gate.ts + ch.d;
    const T* pz = kZ ? in.z.p + b * in.z.bs + t0 * in.z.ts + ch.d : nullptr;
    uint32_t g[kRun];
    if (m == kRun) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) g[i] = W::load(pg + i * in.gate.ts, ch.have);
#pragma unroll
      for (int i = 0; i < kRun; ++i) x[i] = W::load(px + i * in.x.ts, ch.have);
      if constexpr (kZ) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) z[i] = W::load(pz + i * in.z.ts, ch.have);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int have = i < m ? ch.have : 0;
        g[i] = W::load(pg + i * in.gate.ts, have);
        x[i] = W::load(px + i * in.x.ts, have);
        if constexpr (kZ) z[i] = W::load(pz + i * in.z.ts, have);
      }
    }
    float L[C], Q[C], P[C], F[C], h[C];
#pragma unroll
    for (int k = 0; k < C; ++k) L[k] = 0.0f, Q[k] = 0.0f, P[k] = 1.0f;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        c[i][k] = i < m ? gate_coef(W::get(g[i], k)) : 0.0f;  // past the end: held
        L[k] = gate_step(c[i][k], L[k], W::get(x[i], k));
        Q[k] = gate_step(c[i][k], Q[k], 1.0f);
        P[k] *= keep(c[i][k]);
      }
    }
#pragma unroll
    for (int k = 0; k < C; ++k) F[k] = map_keep(Q[k], P[k]);
    join_runs<C, false>(joints, turn, rank, blocks, L, F, carry, h);
    if (out.checkpoints != nullptr && m > 0) {
      float* p = out.checkpoints + (b * out.n_check + t0 / kRun) * in.dim;
#pragma unroll
      for (int k = 0; k < C; ++k)
        if (k < ch.have) p[ch.at(k)] = h[k];
    }
    T* py = out.y + b * out.ybs + t0 * out.yts + ch.d;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      float o[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        h[k] = gate_step(c[i][k], h[k], W::get(x[i], k));
        o[k] = h[k];
        if constexpr (kZ) {
          const float v = W::get(z[i], k);
          o[k] *= v * sigmoid(v);
        }
      }
      if (i < m) W::store(py + i * out.yts, ch.have, o);
    }
  }
  if (out.final_state != nullptr && rank == 0 && warp == 0) {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (k < ch.have) out.final_state[b * in.dim + ch.at(k)] = carry[k];
  }
  // past the sequence's end
  const float zero[C] = {};
  for (int64_t t = n + rank * kGateWarps + warp; t < in.len; t += blocks * kGateWarps)
    W::store(out.y + b * out.ybs + t * out.yts + ch.d, ch.have, zero);
  cooperative_groups::this_cluster().sync();  // others write here
}

template <class T>
struct GateOut {
  T *dx, *dgate, *dz;  // contiguous
  float* dstate;
};

template <class T, bool kZ, bool kWide>
__global__ void __launch_bounds__(kGateWarps * 32, 2)
gated_scan_backward_kernel(GateIn<T> in, Strided<T> dy, const float* __restrict__ dfinal,
                           const float* __restrict__ checkpoints, int64_t n_check, GateOut<T> out,
                           int blocks) {
  constexpr int C = Lane<T>::C;
  using W = Word<T, kWide>;
  __shared__ Joints<C> joints;
  const int warp = threadIdx.x / 32;
  const int rank = (int)(blockIdx.x % (unsigned)blocks);
  const int64_t per = (in.dim + 32 * C - 1) / (32 * C);
  int64_t group;
  const int64_t b = divide(blockIdx.x / (unsigned)blocks, per, group);
  const Channels<T, kWide> ch(group, in.dim);
  const int64_t n = sequence_length(in.lengths, in.index_bytes, b, in.len);
  float carry[C];  // a[t+1] G[t+1]
#pragma unroll
  for (int k = 0; k < C; ++k)
    carry[k] = dfinal != nullptr && k < ch.have ? dfinal[b * in.dim + ch.at(k)] : 0.0f;
  const int64_t step = (int64_t)blocks * kTileSteps;
  int turn = 0;
  for (int64_t s0 = (n + step - 1) / step * step - step; s0 >= 0; s0 -= step, turn ^= 1) {
    const int64_t t0 = s0 + (int64_t)rank * kTileSteps + warp * kRun;
    const int m = (int)max((int64_t)0, min((int64_t)kRun, n - t0));
    uint32_t x[kRun], g[kRun], z[kRun], e[kRun];
    const T* px = in.x.p + b * in.x.bs + t0 * in.x.ts + ch.d;
    const T* pg = in.gate.p + b * in.gate.bs + t0 * in.gate.ts + ch.d;
    const T* pz = kZ ? in.z.p + b * in.z.bs + t0 * in.z.ts + ch.d : nullptr;
    const T* pe = dy.p + b * dy.bs + t0 * dy.ts + ch.d;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int have = i < m ? ch.have : 0;
      g[i] = W::load(pg + i * in.gate.ts, have);
      x[i] = W::load(px + i * in.x.ts, have);
      e[i] = W::load(pe + i * dy.ts, have);
      if constexpr (kZ) z[i] = W::load(pz + i * in.z.ts, have);
    }
    float h[C];
    {
      const float* p = checkpoints + (b * n_check + t0 / kRun) * in.dim;
#pragma unroll
      for (int k = 0; k < C; ++k) h[k] = m > 0 && k < ch.have ? p[ch.at(k)] : 0.0f;
    }
    // the states again; what the way back takes of each step
    float c[kRun][C], d[kRun][C], v[kRun][C];
    const int64_t at = (b * in.len + t0) * in.dim + ch.d;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      float o[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const float xv = W::get(x[i], k);
        c[i][k] = i < m ? gate_coef(W::get(g[i], k)) : 0.0f;
        d[i][k] = h[k] - xv;
        h[k] = gate_step(c[i][k], h[k], xv);
        v[i][k] = W::get(e[i], k);
        if constexpr (kZ) {
          const float q = W::get(z[i], k), s = sigmoid(q);
          o[k] = v[i][k] * h[k] * (s * (1.0f + q * (1.0f - s)));
          v[i][k] *= q * s;
        }
      }
      if constexpr (kZ) {
        if (i < m) W::store(out.dz + at + i * in.dim, ch.have, o);
      }
    }
    float L[C], Q[C], P[C], F[C], B[C];
#pragma unroll
    for (int k = 0; k < C; ++k) L[k] = 0.0f, Q[k] = 0.0f, P[k] = 1.0f;
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        L[k] = forget(c[i][k], L[k] + v[i][k]);
        Q[k] = gate_step(c[i][k], Q[k], 1.0f);
        P[k] *= keep(c[i][k]);
      }
    }
#pragma unroll
    for (int k = 0; k < C; ++k) F[k] = map_keep(Q[k], P[k]);
    join_runs<C, true>(joints, turn, rank, blocks, L, F, carry, B);
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i) {
      float o[C], p[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const float G = B[k] + v[i][k], a = fabsf(c[i][k]);
        o[k] = take(c[i][k]) * G;
        p[k] = d[i][k] * G * (a * (1.0f - a));
        B[k] = forget(c[i][k], G);
      }
      if (i < m) {
        W::store(out.dx + at + i * in.dim, ch.have, o);
        W::store(out.dgate + at + i * in.dim, ch.have, p);
      }
    }
  }
  if (out.dstate != nullptr && rank == 0 && warp == 0) {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (k < ch.have) out.dstate[b * in.dim + ch.at(k)] = carry[k];
  }
  const float zero[C] = {};
  for (int64_t t = n + rank * kGateWarps + warp; t < in.len; t += blocks * kGateWarps) {
    const int64_t at = (b * in.len + t) * in.dim + ch.d;
    W::store(out.dx + at, ch.have, zero);
    W::store(out.dgate + at, ch.have, zero);
    if constexpr (kZ) W::store(out.dz + at, ch.have, zero);
  }
  cooperative_groups::this_cluster().sync();
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

// Blocks that share a sequence's time.
#ifndef CR_GATE_BLOCKS
#define CR_GATE_BLOCKS 304
#endif
int gate_blocks(int64_t groups, int64_t len) {
  int c = 1;
  while (c < kMostCluster && groups * c * 2 <= CR_GATE_BLOCKS && (int64_t)c * kTileSteps < len) c *= 2;
  return c;
}

template <class... P, class... A>
void launch_clusters(void (*kernel)(P...), int64_t blocks, int cluster, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kGateWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  if (cluster > 8 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess)
    return;
  cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The kernel for a call with z or without, and for rows of whole words or any.
// (For binary32 a word is a channel.)
#define CR_GATE_KERNEL(NAME, T, Z, WIDE)                                      \
  (Z ? WIDE ? NAME<T, true, true> : NAME<T, true, sizeof(T) == 4>             \
     : WIDE ? NAME<T, false, true> : NAME<T, false, sizeof(T) == 4>)

template <class T>
bool gate_wide(const cr_gated_scan_args* a) {
  if (sizeof(T) == 4) return true;
  const size_t es = sizeof(T);
  return a->dim % 2 == 0 && rows_aligned(a->x, a->x_batch_stride, a->x_time_stride, es, 4) &&
         rows_aligned(a->gate, a->gate_batch_stride, a->gate_time_stride, es, 4) &&
         (a->z == nullptr || rows_aligned(a->z, a->z_batch_stride, a->z_time_stride, es, 4));
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
  const int64_t per = ceil_div(a->dim, 128 / (int64_t)es);
  if (a->batch > kMaxBlocks / kMostCluster / per) return CR_ERR_UNSUPPORTED;
  const int c = gate_blocks(a->batch * per, a->len);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    const GateFwd<T> out = {static_cast<T*>(y), y_batch_stride, y_time_stride, final_state,
                            checkpoints, cr_gated_scan_checkpoints(a->len)};
    const bool wide = gate_wide<T>(a) &&
                      (es == 4 || rows_aligned(y, y_batch_stride, y_time_stride, es, 4));
    auto kernel = CR_GATE_KERNEL(gated_scan_kernel, T, (a->z != nullptr), wide);
    CR_LAUNCH(kKGatedScan, s,
              launch_clusters(kernel, a->batch * per * c, c, s, gate_in<T>(a), out, c));
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
  const int64_t per = ceil_div(a->dim, 128 / (int64_t)es);
  if (a->batch > kMaxBlocks / kMostCluster / per) return CR_ERR_UNSUPPORTED;
  const int c = gate_blocks(a->batch * per, a->len);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    const Strided<T> dy = {static_cast<const T*>(g->dy), g->dy_batch_stride, g->dy_time_stride};
    const GateOut<T> out = {static_cast<T*>(g->dx), static_cast<T*>(g->dgate),
                            static_cast<T*>(g->dz), g->dstate};
    const bool wide =
        gate_wide<T>(a) &&
        (es == 4 || (rows_aligned(g->dy, g->dy_batch_stride, g->dy_time_stride, es, 4) &&
                     ptr_aligned(g->dx, 4) && ptr_aligned(g->dgate, 4) && ptr_aligned(g->dz, 4)));
    auto kernel = CR_GATE_KERNEL(gated_scan_backward_kernel, T, (a->z != nullptr), wide);
    CR_LAUNCH(kKGatedScanBackward, s,
              launch_clusters(kernel, a->batch * per * c, c, s, gate_in<T>(a), dy, g->dfinal,
                              g->checkpoints, cr_gated_scan_checkpoints(a->len), out, c));
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
