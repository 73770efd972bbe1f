// Shared by the selective state space scan (cr_selective_scan.cu) and its
// gradient (cr_selective_scan_backward.cu).
//
//   delta[t] = softplus(dt[t] + dt_bias)
//   h[t,n]   = a[t,n] h[t-1,n] + delta[t] u[t] B[t,n],   a = exp(delta[t] A[n])
//   y[t]     = (sum_n C[t,n] h[t,n] + D u[t]) silu(z[t])
// backward, with p[t] = dy[t] silu(z[t]):
//   g[t,n]   = C[t,n] p[t] + a[t+1,n] g[t+1,n]
//   dC[t,n]  = sum_d p h,  dB[t,n] = sum_d g delta u,  q = g a h[t-1]
//   ddelta   = sum_n q A + u sum_n g B,  du = delta sum_n g B + D p
//   dA = sum q delta,  dD = sum p u,  dz = dy (C.h + D u) silu'(z)
//
// G lanes share a channel, four states each; a warp holds 32 / G channels.
#pragma once

#include <algorithm>
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {  // each file its own

constexpr int kS = 4;            // states a lane
constexpr int kScanThreads = 128;
constexpr int kCheckpoint = 16;  // steps between checkpoints

// What every kernel of a call reads.
template <class T>
struct ScanIn {
  int64_t batch, len, dim, group_dim;
  int N, groups;
  bool softplus;
  const T *u, *dt, *z, *B, *C;
  int64_t ubs, uts, dbs, dts, zbs, zts, Bbs, Bts, Cbs, Cts;
  const float *A, *D, *dt_bias, *state;
  const void* lengths;
  int index_bytes;
};

template <class T>
__device__ __forceinline__ void load_states(const T* p, int n0, int N, float (&f)[kS]) {
#pragma unroll
  for (int k = 0; k < kS; ++k) f[k] = n0 + k < N ? to_f32(p[n0 + k]) : 0.0f;
}

// A lane's states in a row of N floats; wide: N % 4 == 0 and 16-byte rows.
__device__ __forceinline__ void read_states(const float* p, int n0, int N, bool wide,
                                            float (&f)[kS]) {
  if (wide && n0 < N) {
    const float4 v = *reinterpret_cast<const float4*>(p + n0);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  } else {
    load_states(p, n0, N, f);
  }
}
__device__ __forceinline__ void store_states(float* p, int n0, int N, bool wide,
                                             const float (&f)[kS]) {
  if (wide) {
    if (n0 < N) *reinterpret_cast<float4*>(p + n0) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int k = 0; k < kS; ++k)
      if (n0 + k < N) p[n0 + k] = f[k];
  }
}

// Lanes of a warp: lane = g (32 / G) + c, so that neighbouring lanes read the
// same B and C (a 16-byte shared load takes 2 cycles where lane pairs agree
// and 4 where they do not).
template <int G>
struct Lanes {
  static constexpr int kChannels = 32 / G;  // of a warp
  __device__ static __forceinline__ int g() { return (threadIdx.x % 32) / kChannels; }
  __device__ static __forceinline__ int c() {
    return threadIdx.x / 32 * kChannels + threadIdx.x % kChannels;
  }
};

// The sum over the G lanes of a channel: as a tree over the bits of g from
// bit 2 upwards, then bit 0, then bit 1. Two pairs of time steps at once: the
// last two levels halve the values instead of repeating them, so that lane g
// ends with step 2 (g & 1) + (g >> 1 & 1) in v[0] (G = 2: a pair in v[0..1],
// G = 1: all four).
template <int G>
__device__ __forceinline__ void sum_lanes4(F2 p0, F2 p1, int g, float (&v)[4]) {
  constexpr int L = 32 / G;
  unpack2(p0, v[0], v[1]);
  unpack2(p1, v[2], v[3]);
#pragma unroll
  for (int s = 4; s < G; s *= 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(~0u, v[i], s * L);
  if (G >= 2) {
    const bool up = g & 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float keep = up ? v[i + 2] : v[i], send = up ? v[i] : v[i + 2];
      v[i] = keep + __shfl_xor_sync(~0u, send, L);
    }
  }
  if (G >= 4) {
    const bool up = g & 2;
    const float keep = up ? v[1] : v[0], send = up ? v[0] : v[1];
    v[0] = keep + __shfl_xor_sync(~0u, send, 2 * L);
  }
}

// The same sum of one value where neighbouring lanes share a channel.
template <int G>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int s = 4; s < G; s *= 2) v += __shfl_xor_sync(~0u, v, s);
#pragma unroll
  for (int s = 1; s < G && s < 4; s *= 2) v += __shfl_xor_sync(~0u, v, s);
  return v;
}

// A block's time tile. The elements of u, dt, z and y are handled by all
// threads, two steps of VE neighbouring channels at a time; the recurrence by
// G lanes a channel, two steps at a time.
template <class T, int G, int kSteps = (G <= 2 ? 16 : 32)>
struct Tile {
  static constexpr int CH = kScanThreads / G;         // channels of a block
  static constexpr int TT = kSteps;                   // steps of a tile
  static constexpr int TP = TT / 2;                   // pairs of steps
  static constexpr int E = TP * CH / kScanThreads;    // pairs a thread
  static constexpr int W = 16 / (int)sizeof(T);
  static constexpr int VE = E < 1 ? 1 : E < W ? E : W;  // channels of an access
  static constexpr int NV = CH / VE;                  // accesses a row
  static constexpr int ACC = TP * NV;                 // accesses of the tile
  static constexpr int NL = (ACC + kScanThreads - 1) / kScanThreads;
  static constexpr int NP = G * kS;                   // states, padded
  static constexpr int ACC_BC = TP * G;
  static constexpr int NBC = (ACC_BC + kScanThreads - 1) / kScanThreads;
  static constexpr int YS = CH + 8;                   // row of the y tile, in floats
  static_assert(TT % kCheckpoint == 0 && kCheckpoint % 4 == 0, "tile");

  // Pair tp of channel c is a quadruple (delta, delta', du, du') of its two
  // steps. The quadruples of an access are permuted within VE, so that eight
  // threads that write at once meet different banks.
  static __device__ __forceinline__ int slot(int tp, int c) {
    constexpr int kGroup = VE < 8 ? 8 / VE : 1;
    return tp * CH + (c ^ (c / VE / kGroup % VE));
  }
};

// A thread's accesses to a tensor's tiles: two rows of V elements each,
// `PER_ROW` accesses a row and ALL a tile. `p` is where the first stands and
// moves on by a tile.
template <class T, int V, int NACC, int ALL, int PER_ROW, bool kWide>
struct Rows {
  const T* p;
  int64_t ts, tile;  // elements between rows and between tiles
  int have;          // elements of the access that exist, at most V
  bool wide;

  // base: row 0 of the sequence at the block's first channel or state
  __device__ __forceinline__ Rows(const T* base, int64_t ts_, int64_t t0, int tile_steps,
                                  int elements, bool wide_) {
    const int c = threadIdx.x % PER_ROW * V;
    p = base + (t0 + threadIdx.x / PER_ROW * 2) * ts_ + c;
    ts = ts_;
    tile = tile_steps * ts_;
    have = min(V, elements - c);
    wide = wide_ && have == V;
  }
  // Reads the next tile into registers; rows at or past `left` are zero and
  // not read.
  __device__ __forceinline__ void load(int left, Raw<T, V, kWide> (&out)[NACC][2]) {
#pragma unroll
    for (int i = 0; i < NACC; ++i) {
      const int t = (i * kScanThreads + threadIdx.x) / PER_ROW * 2;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (t + j < left && (ALL % kScanThreads == 0 || i * kScanThreads + threadIdx.x < ALL))
          out[i][j].load(p + (i * (kScanThreads / PER_ROW) * 2 + j) * ts, wide, have);
        else
          out[i][j].zero();
      }
    }
    p += tile;
  }
};

// B or C as pairs of steps: quadruples (n, n', n + 1, n' + 1).
template <class TL, class T, bool kWide>
__device__ __forceinline__ void tile_put_states(const Raw<T, kS, kWide> (&in)[TL::NBC][2],
                                                float4* tile) {
#pragma unroll
  for (int i = 0; i < TL::NBC; ++i) {
    const int idx = i * kScanThreads + threadIdx.x;
    if (idx < TL::ACC_BC) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        tile[idx * 2 + k] = make_float4(in[i][0].get(2 * k), in[i][1].get(2 * k),
                                        in[i][0].get(2 * k + 1), in[i][1].get(2 * k + 1));
    }
  }
}

// Two steps of a lane's four states: h' = a h + du B with a = exp2(delta A),
// A holding log2(e) A twice, and where C is given the pair of C.h (a chain
// over the four states).
template <bool kDot>
__device__ __forceinline__ F2 lane_steps(const F2 (&A)[kS], float (&h)[kS], const float4& e4,
                                         const float4 (&Bq)[2], const float4 (&Cq)[2]) {
  const F2 delta = pack2(e4.x, e4.y), du = pack2(e4.z, e4.w);
  F2 p = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 B = Bq[j];
    const float4 C = kDot ? Cq[j] : B;
    const F2 Bn[2] = {pack2(B.x, B.y), pack2(B.z, B.w)};
    const F2 Cn[2] = {pack2(C.x, C.y), pack2(C.z, C.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = 2 * j + i;
      float x0, x1, b0, b1;
      unpack2(mul2(delta, A[n]), x0, x1);
      unpack2(mul2(du, Bn[i]), b0, b1);
      const float h0 = fmaf(exp2_fast(x0), h[n], b0);
      h[n] = fmaf(exp2_fast(x1), h0, b1);
      if (kDot) p = n == 0 ? mul2(Cn[i], pack2(h0, h[n])) : fma2(Cn[i], pack2(h0, h[n]), p);
    }
  }
  return p;
}

// Lanes that share a channel of N states.
[[maybe_unused]] int scan_lanes(int N) {
  int g = 1;
  while (g * kS < N) g *= 2;
  return g;
}

// Blocks of a call of (batch, dim) with G lanes a channel; 0 if too many.
[[maybe_unused]] int64_t scan_blocks(int64_t batch, int64_t dim, int groups, int G) {
  const int64_t per_group = ceil_div(dim / groups, kScanThreads / G);
  const int64_t all = per_group * groups;
  return all > kMaxBlocks / (batch > 0 ? batch : 1) ? 0 : all * batch;
}

// The checks that all calls share.
[[maybe_unused]] cr_status check_scan(const cr_selective_scan_args* a, bool step) {
  if (a == nullptr) return CR_ERR_INVALID_ARG;
  const size_t es = model_esize(a->dt_type);
  if (es == 0 || a->batch < 0 || a->len < 0 || a->dim < 0 || a->dstate < 1 || a->groups < 1 ||
      a->reserved != 0 || (a->softplus != 0 && a->softplus != 1) || a->dim % a->groups != 0)
    return CR_ERR_INVALID_ARG;
  if (step && a->len != 1) return CR_ERR_INVALID_ARG;
  if (a->dstate > 128) return CR_ERR_UNSUPPORTED;
  const int64_t strides[10] = {a->u_batch_stride, a->u_time_stride, a->dt_batch_stride,
                               a->dt_time_stride, a->z_batch_stride, a->z_time_stride,
                               a->B_batch_stride, a->B_time_stride, a->C_batch_stride,
                               a->C_time_stride};
  for (int64_t v : strides)
    if (v < 0) return CR_ERR_INVALID_ARG;
  if (a->lengths != nullptr && !step &&
      (!index_width_ok(a->index_bytes) || !ptr_aligned(a->lengths, a->index_bytes)))
    return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->dim > 0) {
    if (a->A == nullptr) return CR_ERR_INVALID_ARG;
    if (a->len > 0 && (a->u == nullptr || a->dt == nullptr || a->B == nullptr || a->C == nullptr))
      return CR_ERR_INVALID_ARG;
    if (scan_blocks(a->batch, a->dim, a->groups, scan_lanes(a->dstate)) == 0)
      return CR_ERR_UNSUPPORTED;
  }
  if (!ptr_aligned(a->u, es) || !ptr_aligned(a->dt, es) || !ptr_aligned(a->z, es) ||
      !ptr_aligned(a->B, es) || !ptr_aligned(a->C, es) || !ptr_aligned(a->A, 4) ||
      !ptr_aligned(a->D, 4) || !ptr_aligned(a->dt_bias, 4) || !ptr_aligned(a->state, 4))
    return CR_ERR_INVALID_ARG;
  return CR_OK;
}

template <class T>
ScanIn<T> scan_in(const cr_selective_scan_args* a) {
  ScanIn<T> in;
  in.batch = a->batch;
  in.len = a->len;
  in.dim = a->dim;
  in.group_dim = a->dim / a->groups;
  in.N = a->dstate;
  in.groups = a->groups;
  in.softplus = a->softplus != 0;
  in.u = static_cast<const T*>(a->u);
  in.dt = static_cast<const T*>(a->dt);
  in.z = static_cast<const T*>(a->z);
  in.B = static_cast<const T*>(a->B);
  in.C = static_cast<const T*>(a->C);
  in.ubs = a->u_batch_stride, in.uts = a->u_time_stride;
  in.dbs = a->dt_batch_stride, in.dts = a->dt_time_stride;
  in.zbs = a->z_batch_stride, in.zts = a->z_time_stride;
  in.Bbs = a->B_batch_stride, in.Bts = a->B_time_stride;
  in.Cbs = a->C_batch_stride, in.Cts = a->C_time_stride;
  in.A = a->A;
  in.D = a->D;
  in.dt_bias = a->dt_bias;
  in.state = a->state;
  in.lengths = a->lengths;
  in.index_bytes = a->index_bytes;
  return in;
}

// Runs BODY with G bound to the lanes a channel takes.
#define CR_SCAN_LANES(LANES, ...)                            \
  switch (LANES) {                                           \
    case 1: { constexpr int G = 1; __VA_ARGS__; break; }     \
    case 2: { constexpr int G = 2; __VA_ARGS__; break; }     \
    case 4: { constexpr int G = 4; __VA_ARGS__; break; }     \
    case 8: { constexpr int G = 8; __VA_ARGS__; break; }     \
    case 16: { constexpr int G = 16; __VA_ARGS__; break; }   \
    default: { constexpr int G = 32; __VA_ARGS__; break; }   \
  }

}  // namespace
}  // namespace cr
