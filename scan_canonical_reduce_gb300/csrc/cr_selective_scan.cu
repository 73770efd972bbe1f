// Selective state space scan, its gradient, and its single-token form.
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
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

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

// A block's channels lie in one group: block i of a sequence is block
// i % per_group of group i / per_group.
struct Place {
  int64_t b, d;
  int group, g, c;
  bool live;
};

template <int G>
__device__ __forceinline__ Place place(int64_t group_dim, int groups) {
  constexpr int CH = kScanThreads / G;
  const int64_t per_group = (group_dim + CH - 1) / CH;
  Place p;
  const int64_t i = blockIdx.x;
  const int64_t blk = i % (per_group * groups);
  p.b = i / (per_group * groups);
  p.group = (int)(blk / per_group);
  p.c = threadIdx.x / G;
  p.g = threadIdx.x % G;
  const int64_t in_group = blk % per_group * CH + p.c;
  p.live = in_group < group_dim;
  p.d = p.group * group_dim + (p.live ? in_group : 0);
  return p;
}

template <class T>
__device__ __forceinline__ void load_states(const T* p, int n0, int N, float (&f)[kS]) {
#pragma unroll
  for (int k = 0; k < kS; ++k) f[k] = n0 + k < N ? to_f32(p[n0 + k]) : 0.0f;
}

// One lane's four states of a channel: decays and states as two pairs.
struct Lane {
  F2 A[2];  // A log2(e)
  F2 h[2];
};

__device__ __forceinline__ void lane_init(Lane& l, const float (&A)[kS], const float (&h)[kS]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    l.A[j] = pack2(A[2 * j] * kLog2e, A[2 * j + 1] * kLog2e);
    l.h[j] = pack2(h[2 * j], h[2 * j + 1]);
  }
}

__device__ __forceinline__ void lane_states(const Lane& l, float (&h)[kS]) {
  unpack2(l.h[0], h[0], h[1]);
  unpack2(l.h[1], h[2], h[3]);
}

// h = exp(delta A) h + (delta u) B, with delta and delta u given twice.
__device__ __forceinline__ void lane_step(Lane& l, F2 delta, F2 du, F2 B0, F2 B1) {
  const F2 B[2] = {B0, B1};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float x0, x1;
    unpack2(mul2(delta, l.A[j]), x0, x1);
    l.h[j] = fma2(pack2(exp2_fast(x0), exp2_fast(x1)), l.h[j], mul2(du, B[j]));
  }
}

// This lane's part of C.h: (C0 h0 + C2 h2) + (C1 h1 + C3 h3).
__device__ __forceinline__ float lane_dot(const Lane& l, F2 C0, F2 C1) {
  float lo, hi;
  unpack2(fma2(C1, l.h[1], mul2(C0, l.h[0])), lo, hi);
  return lo + hi;
}

// The sum over the G lanes of a channel: lanes g, g + 4, g + 8, ... first,
// which leaves four partial sums, then (p0 + p1) + (p2 + p3).
template <int G>
__device__ __forceinline__ float partial_lanes(float v) {
#pragma unroll
  for (int s = 4; s < G; s *= 2) v += __shfl_xor_sync(~0u, v, s);
  return v;
}

template <int G>
__device__ __forceinline__ float sum_lanes(float v) {
  v = partial_lanes<G>(v);
#pragma unroll
  for (int s = 1; s < G && s < 4; s *= 2) v += __shfl_xor_sync(~0u, v, s);
  return v;
}

template <int G>
__device__ __forceinline__ float sum_partials(float4 p) {
  return G == 1 ? p.x : G == 2 ? p.x + p.y : (p.x + p.y) + (p.z + p.w);
}

// A block's time tile. The elements of u, dt, z and y are handled by all
// threads, VE neighbouring channels at a time; the recurrence by G lanes a
// channel.
template <class T, int G>
struct Tile {
  static constexpr int CH = kScanThreads / G;        // channels of a block
  static constexpr int TT = G <= 2 ? 16 : 32;        // steps of a tile
  static constexpr int E = TT * CH / kScanThreads;   // elements a thread
  static constexpr int W = 16 / (int)sizeof(T);
  static constexpr int VE = E < W ? E : W;           // channels of an access
  static constexpr int NV = CH / VE;                 // accesses a row
  static constexpr int NL = E / VE;                  // accesses a thread
  static constexpr int NP = G * kS;                  // states, padded
  static constexpr int NBC = (TT * G + kScanThreads - 1) / kScanThreads;
  static_assert(TT % 4 == 0 && kCheckpoint % 4 == 0 && TT % kCheckpoint == 0, "tile");

  // Element (t, c) of the tile is a quadruple of floats: (delta, delta, du,
  // du) for the recurrence, then the partial sums of y. The quadruples of an
  // access are permuted so that the threads that write at once, and the lanes
  // that read a step, meet different banks: quadruple k of access v in row t
  // is at (t CH + v VE + k) ^ f, f < VE.
  static __device__ __forceinline__ int flip(int t, int v) {
    const int i = t * NV + v;
    return VE == 8 ? (i & 7) : VE == 4 ? (i >> 1 & 3) : 0;
  }
  static __device__ __forceinline__ int slot(int t, int c) {
    return t * CH + (c ^ flip(t, c / VE));
  }
};

// A tensor's rows as accesses of a tile see them.
template <class T>
struct Rows {
  const T* p;   // row 0 of the sequence at the block's first channel
  int64_t ts;
  bool wide;
};

// Reads rows [t0, t0 + TT) of the tile into registers; rows at or past `end`
// are zero and not read.
template <class TL, class T>
__device__ __forceinline__ void tile_load(const Rows<T>& r, int64_t t0, int64_t end, int channels,
                                          Raw<T, TL::VE> (&out)[TL::NL]) {
#pragma unroll
  for (int i = 0; i < TL::NL; ++i) {
    const int idx = i * kScanThreads + threadIdx.x;
    const int64_t t = t0 + idx / TL::NV;
    const int c = idx % TL::NV * TL::VE;
    if (t < end)
      out[i].load(r.p + t * r.ts + c, r.wide && c + TL::VE <= channels, channels - c);
    else
      out[i].zero();
  }
}

// The same for B or C: four states of a step at a time.
template <class TL, class T>
__device__ __forceinline__ void tile_load_states(const Rows<T>& r, int64_t t0, int64_t end, int N,
                                                 Raw<T, kS> (&out)[TL::NBC]) {
  constexpr int G = TL::NP / kS;
#pragma unroll
  for (int i = 0; i < TL::NBC; ++i) {
    const int idx = i * kScanThreads + threadIdx.x;
    const int64_t t = t0 + idx / G;
    const int n = idx % G * kS;
    if (idx < TL::TT * G && t < end)
      out[i].load(r.p + t * r.ts + n, r.wide && n + kS <= N, N - n);
    else
      out[i].zero();
  }
}

template <class TL, class T>
__device__ __forceinline__ void tile_put_states(const Raw<T, kS> (&in)[TL::NBC], float* tile) {
  constexpr int G = TL::NP / kS;
#pragma unroll
  for (int i = 0; i < TL::NBC; ++i) {
    const int idx = i * kScanThreads + threadIdx.x;
    if (idx < TL::TT * G)
      reinterpret_cast<float4*>(tile)[idx] =
          make_float4(in[i].get(0), in[i].get(1), in[i].get(2), in[i].get(3));
  }
}

// Sequences with few channels are cut into segments that run side by side:
// a first launch (kStates) takes every segment but the last from a zero state
// to its end and its sum of delta, the second starts a segment from the
// state that these give, H' = exp(A sum delta) H + E in segment order.
struct Segments {
  int64_t count, len;
  float* E;     // [count - 1][batch][dim][NP]
  float* sum;   // [count - 1][batch][dim]
};

template <class T>
struct ScanOut {
  T* y;
  int64_t ybs, yts;
  float* final_state;
  float* checkpoints;
  int64_t n_check;
  bool wide, wide_y, wide_BC;
};

#ifndef CR_SCAN_BLOCKS
#define CR_SCAN_BLOCKS 4
#endif
template <class T, int G, bool kStates>
__global__ void __launch_bounds__(kScanThreads, CR_SCAN_BLOCKS)
selective_scan_kernel(ScanIn<T> in, ScanOut<T> out, Segments sg) {
  using TL = Tile<T, G>;
  __shared__ float4 dd[TL::TT * TL::CH];
  __shared__ __align__(16) float Bs[TL::TT * TL::NP];
  __shared__ __align__(16) float Cs[kStates ? 4 : TL::TT * TL::NP];
  __shared__ __align__(16) float Ds[TL::CH], biases[TL::CH];

  const int tid = threadIdx.x, g = tid % G, c = tid / G, n0 = g * kS;
  const int64_t per_group = (in.group_dim + TL::CH - 1) / TL::CH;
  int64_t i = blockIdx.x;
  const int64_t blk = i % (per_group * in.groups);
  i /= per_group * in.groups;
  const int64_t seg = i % (kStates ? sg.count - 1 : sg.count), b = i / (kStates ? sg.count - 1 : sg.count);
  const int64_t group = blk / per_group, first = blk % per_group * TL::CH;
  const int channels = (int)min((int64_t)TL::CH, in.group_dim - first);
  const int64_t d0 = group * in.group_dim + first;
  const bool live = c < channels;
  const int64_t d = d0 + (live ? c : 0);
  const int64_t len = sequence_length(in.lengths, in.index_bytes, b, in.len);
  const int64_t begin = seg * sg.len, end = min(in.len, begin + sg.len), stop = min(len, end);

  if (tid < TL::CH) {
    Ds[tid] = (in.D != nullptr && tid < channels) ? in.D[d0 + tid] : 0.0f;
    biases[tid] = (in.dt_bias != nullptr && tid < channels) ? in.dt_bias[d0 + tid] : 0.0f;
  }
  Lane l;
  {
    float A[kS], h[kS] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_states(in.A + d * in.N, n0, in.N, A);
    if (!kStates && in.state != nullptr)
      load_states(in.state + (b * in.dim + d) * in.N, n0, in.N, h);
    lane_init(l, A, h);
    if (!kStates) {
      const float* E = sg.E + (b * in.dim + d) * TL::NP + n0;
      const float* sum = sg.sum + b * in.dim + d;
#pragma unroll 4
      for (int64_t s = 0; s < seg; ++s) {
        const float4 e = *reinterpret_cast<const float4*>(E + s * in.batch * in.dim * TL::NP);
        const float x = sum[s * in.batch * in.dim];
        const F2 ee[2] = {pack2(e.x, e.y), pack2(e.z, e.w)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x0, x1;
          unpack2(mul2(pack2(x, x), l.A[j]), x0, x1);
          l.h[j] = fma2(pack2(exp2_fast(x0), exp2_fast(x1)), l.h[j], ee[j]);
        }
      }
    }
  }

  const Rows<T> ru = {in.u + b * in.ubs + d0, in.uts, out.wide};
  const Rows<T> rd = {in.dt + b * in.dbs + d0, in.dts, out.wide};
  const Rows<T> rz = {in.z + b * in.zbs + d0, in.zts, out.wide};
  const Rows<T> rB = {in.B + b * in.Bbs + group * in.N, in.Bts, out.wide_BC};
  const Rows<T> rC = {in.C + b * in.Cbs + group * in.N, in.Cts, out.wide_BC};
  const bool gated = !kStates && in.z != nullptr;
  Raw<T, TL::VE> pu[TL::NL], pd[TL::NL], pz[TL::NL];
  Raw<T, kS> pB[TL::NBC], pC[TL::NBC];
  auto load = [&](int64_t t0) {
    tile_load<TL>(ru, t0, stop, channels, pu);
    tile_load<TL>(rd, t0, stop, channels, pd);
    if (gated) tile_load<TL>(rz, t0, stop, channels, pz);
    tile_load_states<TL>(rB, t0, stop, in.N, pB);
    if (!kStates) tile_load_states<TL>(rC, t0, stop, in.N, pC);
  };
  load(begin);
  __syncthreads();  // Ds, biases
  float total = 0.0f;

  int64_t t0 = begin;
  for (; t0 < stop; t0 += TL::TT) {
    // elements: delta and delta u into the tile; u and z stay for the end
    Raw<T, TL::VE> ku[TL::NL], kz[TL::NL];
#pragma unroll
    for (int i = 0; i < TL::NL; ++i) {
      const int idx = i * kScanThreads + tid, t = idx / TL::NV, c0 = idx % TL::NV * TL::VE;
      const bool in_seq = t0 + t < stop;
      const int at = TL::slot(t, c0) * 16;
      float delta[TL::VE];
#pragma unroll
      for (int k = 0; k < TL::VE; ++k) delta[k] = pd[i].get(k) + biases[c0 + k];
      if (in.softplus) {
#pragma unroll
        for (int k = 0; k < TL::VE; ++k) delta[k] = softplus(delta[k]);
      }
#pragma unroll
      for (int k = 0; k < TL::VE; ++k) {
        const float dt = in_seq ? delta[k] : 0.0f;
        const float du = dt * pu[i].get(k);
        *reinterpret_cast<float4*>(reinterpret_cast<char*>(dd) + (at ^ (k * 16))) =
            make_float4(dt, dt, du, du);
      }
      if (!kStates) ku[i] = pu[i];
      if (gated) kz[i] = pz[i];
    }
    tile_put_states<TL>(pB, Bs);
    if (!kStates) tile_put_states<TL>(pC, Cs);
    __syncthreads();
    if (t0 + TL::TT < stop) load(t0 + TL::TT);

    // recurrence
#pragma unroll 2
    for (int t4 = 0; t4 < TL::TT / 4; ++t4) {
      const int t = t4 * 4;
      if (!kStates && out.checkpoints != nullptr && t % kCheckpoint == 0 && live &&
          t0 + t < end) {
        float h[kS];
        lane_states(l, h);
        float* q = out.checkpoints +
                   ((b * out.n_check + (t0 + t) / kCheckpoint) * in.dim + d) * in.N + n0;
#pragma unroll
        for (int k = 0; k < kS; ++k)
          if (n0 + k < in.N) q[k] = h[k];
      }
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const ulonglong2 e = reinterpret_cast<const ulonglong2*>(dd)[TL::slot(t + k, c)];
        const ulonglong2 B = reinterpret_cast<const ulonglong2*>(Bs)[(t + k) * G + g];
        lane_step(l, e.x, e.y, B.x, B.y);
        if (!kStates) {
          const ulonglong2 C = reinterpret_cast<const ulonglong2*>(Cs)[(t + k) * G + g];
          v[k] = partial_lanes<G>(lane_dot(l, C.x, C.y));
        } else {
          float a, a2;
          unpack2(e.x, a, a2);
          total += a;
        }
      }
      if (!kStates) {
        __syncwarp();  // the lanes of a channel have read what they overwrite
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (G <= 4 || g < 4) reinterpret_cast<float*>(dd)[TL::slot(t + k, c) * 4 + g] = v[k];
      }
    }
    __syncthreads();

    // elements: D u, the gate, and out
    if (!kStates) {
#pragma unroll
      for (int i = 0; i < TL::NL; ++i) {
        const int idx = i * kScanThreads + tid, t = idx / TL::NV, c0 = idx % TL::NV * TL::VE;
        const int at = TL::slot(t, c0) * 16;
        float f[TL::VE];
        const bool in_seq = t0 + t < stop;
#pragma unroll
        for (int k = 0; k < TL::VE; ++k) {
          const float4 p = *reinterpret_cast<const float4*>(reinterpret_cast<const char*>(dd) +
                                                            (at ^ (k * 16)));
          float v = fmaf(Ds[c0 + k], ku[i].get(k), sum_partials<G>(p));
          if (gated) {
            const float z = kz[i].get(k);
            v *= z * sigmoid(z);
          }
          f[k] = in_seq ? v : 0.0f;
        }
        const int have = min(TL::VE, channels - c0);
        if (t0 + t < end && have > 0)
          store_f32<T, TL::VE>(out.y + b * out.ybs + (t0 + t) * out.yts + d0 + c0,
                               out.wide_y && have == TL::VE, have, f);
      }
    }
  }
  if (kStates) {
    if (live) {
      float h[kS];
      lane_states(l, h);
      const int64_t row = (seg * in.batch + b) * in.dim + d;
      *reinterpret_cast<float4*>(sg.E + row * TL::NP + n0) = make_float4(h[0], h[1], h[2], h[3]);
      if (g == 0) sg.sum[row] = total;
    }
    return;
  }
  for (; t0 < end; t0 += TL::TT) {  // past the sequence's length
#pragma unroll
    for (int i = 0; i < TL::NL; ++i) {
      const int idx = i * kScanThreads + tid, t = idx / TL::NV, c0 = idx % TL::NV * TL::VE;
      const int have = min(TL::VE, channels - c0);
      float f[TL::VE];
#pragma unroll
      for (int k = 0; k < TL::VE; ++k) f[k] = 0.0f;
      if (t0 + t < end && have > 0)
        store_f32<T, TL::VE>(out.y + b * out.ybs + (t0 + t) * out.yts + d0 + c0,
                             out.wide_y && have == TL::VE, have, f);
    }
  }
  if (out.final_state != nullptr && seg == sg.count - 1 && live) {
    float h[kS];
    lane_states(l, h);
#pragma unroll
    for (int k = 0; k < kS; ++k)
      if (n0 + k < in.N) out.final_state[(b * in.dim + d) * in.N + n0 + k] = h[k];
  }
}

template <class T>
struct ScanBack {
  const T* dy;
  int64_t dybs, dyts;
  const float* dfinal;
  const float* checkpoints;
  T *du, *ddt, *dz;
  float* dstate;
  float* part_BC;  // [batch][len][groups][warps][2][G kS]
  float* part_A;   // [batch][dim][N + 2]: dA, dD, ddt_bias
  int64_t warps;   // a group's, of a sequence
};

template <class T, int G>
__global__ void __launch_bounds__(kScanThreads)
selective_scan_backward_kernel(ScanIn<T> in, ScanBack<T> o, int64_t n_check) {
  constexpr int NP = G * kS;
  const Place p = place<G>(in.group_dim, in.groups);
  const int n0 = p.g * kS;
  const int64_t len = sequence_length(in.lengths, in.index_bytes, p.b, in.len);
  const int64_t row = (p.b * in.dim + p.d) * in.N;
  const int64_t per_group = (in.group_dim + kScanThreads / G - 1) / (kScanThreads / G);
  const int64_t warp =
      (blockIdx.x % (per_group * in.groups)) % per_group * (kScanThreads / 32) + threadIdx.x / 32;
  float A[kS], carry[kS], dA[kS];
  load_states(in.A + p.d * in.N, n0, in.N, A);
#pragma unroll
  for (int k = 0; k < kS; ++k) carry[k] = dA[k] = 0.0f;
  if (o.dfinal != nullptr) load_states(o.dfinal + row, n0, in.N, carry);
  const float Dd = in.D != nullptr ? in.D[p.d] : 0.0f;
  const float bias = in.dt_bias != nullptr ? in.dt_bias[p.d] : 0.0f;
  float dD = 0.0f, dbias = 0.0f;
  const int64_t chunks = (in.len + kCheckpoint - 1) / kCheckpoint;
  for (int64_t ch = chunks - 1; ch >= 0; --ch) {
    const int64_t t0 = ch * kCheckpoint;
    float h[kCheckpoint + 1][kS];
    load_states(o.checkpoints + ((p.b * n_check + ch) * in.dim + p.d) * in.N, n0, in.N, h[0]);
#pragma unroll
    for (int i = 0; i < kCheckpoint; ++i) {
      const int64_t t = t0 + i;
#pragma unroll
      for (int k = 0; k < kS; ++k) h[i + 1][k] = h[i][k];
      if (t < len) {
        float B[kS];
        load_states(in.B + p.b * in.Bbs + t * in.Bts + (int64_t)p.group * in.N, n0, in.N, B);
        const float u = to_f32(in.u[p.b * in.ubs + t * in.uts + p.d]);
        float delta = to_f32(in.dt[p.b * in.dbs + t * in.dts + p.d]) + bias;
        if (in.softplus) delta = softplus(delta);
#pragma unroll
        for (int k = 0; k < kS; ++k)
          h[i + 1][k] = fmaf(exp2_fast(delta * (A[k] * kLog2e)), h[i][k], delta * u * B[k]);
      }
    }
#pragma unroll
    for (int i = kCheckpoint - 1; i >= 0; --i) {
      const int64_t t = t0 + i;
      if (t >= in.len) continue;
      float dB[kS] = {0.0f, 0.0f, 0.0f, 0.0f}, dC[kS] = {0.0f, 0.0f, 0.0f, 0.0f};
      float du = 0.0f, ddt = 0.0f, dz = 0.0f;
      if (t < len) {
        float B[kS], C[kS];
        load_states(in.B + p.b * in.Bbs + t * in.Bts + (int64_t)p.group * in.N, n0, in.N, B);
        load_states(in.C + p.b * in.Cbs + t * in.Cts + (int64_t)p.group * in.N, n0, in.N, C);
        const float u = to_f32(in.u[p.b * in.ubs + t * in.uts + p.d]);
        const float raw = to_f32(in.dt[p.b * in.dbs + t * in.dts + p.d]) + bias;
        const float delta = in.softplus ? softplus(raw) : raw;
        float pt = to_f32(o.dy[p.b * o.dybs + t * o.dyts + p.d]);
        if (in.z != nullptr) {
          const float z = to_f32(in.z[p.b * in.zbs + t * in.zts + p.d]);
          const float s = sigmoid(z);
          float yv = 0.0f;
#pragma unroll
          for (int k = 0; k < kS; ++k) yv = fmaf(C[k], h[i + 1][k], yv);
          yv = fmaf(Dd, u, sum_lanes<G>(yv));
          dz = pt * yv * (s * fmaf(z, 1.0f - s, 1.0f));
          pt *= z * s;
        }
        float gB = 0.0f, qA = 0.0f;
#pragma unroll
        for (int k = 0; k < kS; ++k) {
          const float g = fmaf(C[k], pt, carry[k]);
          dC[k] = pt * h[i + 1][k];
          dB[k] = g * (delta * u);
          gB = fmaf(g, B[k], gB);
          carry[k] = g * exp2_fast(delta * (A[k] * kLog2e));
          const float q = carry[k] * h[i][k];
          dA[k] = fmaf(q, delta, dA[k]);
          qA = fmaf(q, A[k], qA);
        }
        gB = sum_lanes<G>(gB);
        qA = sum_lanes<G>(qA);
        du = fmaf(delta, gB, Dd * pt);
        ddt = fmaf(u, gB, qA);
        if (in.softplus) ddt *= sigmoid(raw);
        dD = fmaf(pt, u, dD);
        dbias += ddt;
      }
      if (p.live && p.g == 0) {
        const int64_t at = (p.b * in.len + t) * in.dim + p.d;
        o.du[at] = from_f32<T>(du);
        o.ddt[at] = from_f32<T>(ddt);
        if (o.dz != nullptr) o.dz[at] = from_f32<T>(dz);
      }
      float* q = o.part_BC + (((p.b * in.len + t) * in.groups + p.group) * o.warps + warp) * 2 * NP;
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        float vB = p.live ? dB[k] : 0.0f, vC = p.live ? dC[k] : 0.0f;
#pragma unroll
        for (int s = G; s < 32; s *= 2) {
          vB += __shfl_xor_sync(~0u, vB, s);
          vC += __shfl_xor_sync(~0u, vC, s);
        }
        if (threadIdx.x % 32 < G) {
          q[n0 + k] = vB;
          q[NP + n0 + k] = vC;
        }
      }
    }
  }
  if (!p.live) return;
  float* q = o.part_A + (p.b * in.dim + p.d) * (in.N + 2);
#pragma unroll
  for (int k = 0; k < kS; ++k) {
    if (n0 + k < in.N) {
      q[n0 + k] = dA[k];
      if (o.dstate != nullptr) o.dstate[row + n0 + k] = carry[k];
    }
  }
  if (p.g == 0) {
    q[in.N] = dD;
    q[in.N + 1] = dbias;
  }
}

// dB and dC: the warps' partials of a (sequence, step, group), in order.
template <class T>
__global__ void __launch_bounds__(kScanThreads)
selective_scan_sum_bc_kernel(const float* __restrict__ part, int64_t rows, int64_t warps, int NP,
                             int N, T* __restrict__ dB, T* __restrict__ dC) {
  const int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= rows * 2 * N) return;
  const int64_t r = i / (2 * N);
  const int j = (int)(i % (2 * N));
  const int which = j / N, n = j % N;
  const float* q = part + r * warps * 2 * NP + which * NP + n;
  float s = 0.0f;
  for (int64_t w = 0; w < warps; ++w) s += q[w * 2 * NP];
  (which ? dC : dB)[r * N + n] = from_f32<T>(s);
}

// dA, dD and ddt_bias: the sequences' partials, in order.
__global__ void __launch_bounds__(kScanThreads)
selective_scan_sum_a_kernel(const float* __restrict__ part, int64_t batch, int64_t dim, int N,
                            float* __restrict__ dA, float* __restrict__ dD,
                            float* __restrict__ dbias) {
  const int64_t n = dim * (N + 2);
  const int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int64_t b = 0; b < batch; ++b) s += part[b * n + i];
  const int64_t d = i / (N + 2);
  const int k = (int)(i % (N + 2));
  if (k < N) dA[d * N + k] = s;
  else if (k == N && dD != nullptr) dD[d] = s;
  else if (k == N + 1 && dbias != nullptr) dbias[d] = s;
}

template <class T, int G>
__global__ void __launch_bounds__(kScanThreads)
selective_scan_step_kernel(ScanIn<T> in, float* __restrict__ state, int64_t state_rows,
                           const void* __restrict__ slots, T* __restrict__ y, int64_t ybs) {
  const Place p = place<G>(in.group_dim, in.groups);
  const int n0 = p.g * kS;
  const int64_t slot = slots != nullptr ? load_index(slots, in.index_bytes, p.b) : p.b;
  float o = 0.0f;
  if (slot >= 0 && slot < state_rows) {  // the same for the whole block
    float* st = state + (slot * in.dim + p.d) * in.N;
    float A[kS], B[kS], C[kS], h[kS] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_states(in.A + p.d * in.N, n0, in.N, A);
    load_states(in.B + p.b * in.Bbs + (int64_t)p.group * in.N, n0, in.N, B);
    load_states(in.C + p.b * in.Cbs + (int64_t)p.group * in.N, n0, in.N, C);
    if (p.live) load_states(st, n0, in.N, h);
    const float u = to_f32(in.u[p.b * in.ubs + p.d]);
    float delta = to_f32(in.dt[p.b * in.dbs + p.d]);
    if (in.dt_bias != nullptr) delta += in.dt_bias[p.d];
    if (in.softplus) delta = softplus(delta);
    const float du = delta * u;
    Lane l;
    lane_init(l, A, h);
    lane_step(l, pack2(delta, delta), pack2(du, du), pack2(B[0], B[1]), pack2(B[2], B[3]));
    const float acc = lane_dot(l, pack2(C[0], C[1]), pack2(C[2], C[3]));
    lane_states(l, h);
    o = fmaf(in.D != nullptr ? in.D[p.d] : 0.0f, u, sum_lanes<G>(acc));
    if (in.z != nullptr) {
      const float z = to_f32(in.z[p.b * in.zbs + p.d]);
      o *= z * sigmoid(z);
    }
    if (p.live) {
#pragma unroll
      for (int k = 0; k < kS; ++k)
        if (n0 + k < in.N) st[n0 + k] = h[k];
    }
  }
  if (p.live && p.g == 0) y[p.b * ybs + p.d] = from_f32<T>(o);
}

int scan_lanes(int N) {
  int g = 1;
  while (g * kS < N) g *= 2;
  return g;
}

// Blocks of a call of (batch, dim) with G lanes a channel; 0 if too many.
int64_t scan_blocks(int64_t batch, int64_t dim, int groups, int G) {
  const int64_t per_group = ceil_div(dim / groups, kScanThreads / G);
  const int64_t all = per_group * groups;
  return all > kMaxBlocks / (batch > 0 ? batch : 1) ? 0 : all * batch;
}

// How a call's sequences are cut. A rule on sizes alone, so that results do
// not depend on the GPU.
#ifndef CR_SCAN_WARPS
#define CR_SCAN_WARPS 2432
#endif
#ifndef CR_SCAN_SPLIT_BELOW
#define CR_SCAN_SPLIT_BELOW 700
#endif
Segments scan_segments(int64_t batch, int64_t len, int64_t dim, int lanes) {
  constexpr int64_t kTile = 32;
  Segments sg;
  sg.E = sg.sum = nullptr;
  sg.count = 1;
  const int64_t warps = batch * ceil_div(dim * lanes, 32);
  if (warps < CR_SCAN_SPLIT_BELOW && warps > 0 && len >= 8 * kTile) {
    sg.count = CR_SCAN_WARPS / warps;
    const int64_t most = len / (4 * kTile);
    if (sg.count > most) sg.count = most;
    if (sg.count > 64) sg.count = 64;
  }
  sg.len = len > 0 ? ceil_div(ceil_div(len, sg.count), kTile) * kTile : kTile;
  sg.count = len > 0 ? ceil_div(len, sg.len) : 1;
  return sg;
}

cr_status check_scan(const cr_selective_scan_args* a, bool step) {
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

extern "C" {

int64_t cr_selective_scan_checkpoints(int64_t len) {
  return len <= 0 ? 0 : cr::ceil_div(len, cr::kCheckpoint);
}

size_t cr_selective_scan_workspace_bytes(int64_t batch, int64_t len, int64_t dim,
                                         int32_t dstate) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || dstate < 1) return 0;
  const int64_t segs = scan_segments(batch, len, dim, scan_lanes(dstate)).count;
  return round256((size_t)(segs - 1) * batch * dim * (scan_lanes(dstate) * kS + 1) * 4) + 256;
}

cr_status cr_selective_scan(const cr_selective_scan_args* a, void* y, int64_t y_batch_stride,
                            int64_t y_time_stride, float* final_state, float* checkpoints,
                            void* ws, size_t ws_bytes, void* stream) {
  using namespace cr;
  const cr_status ok = check_scan(a, false);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt_type);
  if (y_batch_stride < 0 || y_time_stride < 0) return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(y, es) || !ptr_aligned(final_state, 4) || !ptr_aligned(checkpoints, 4))
    return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->dim > 0 && a->len > 0 &&
      (y == nullptr || y == a->u || y == a->dt || y == a->z ||
       (a->len > 1 && y_time_stride < a->dim) || (a->batch > 1 && y_batch_stride < a->dim)))
    return CR_ERR_INVALID_ARG;
  const size_t need =
      cr_selective_scan_workspace_bytes(a->batch, a->len, a->dim, a->dstate);
  if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < need) return CR_ERR_WORKSPACE;
  if (a->batch == 0 || a->dim == 0) return CR_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int lanes = scan_lanes(a->dstate);
  const int64_t blocks = scan_blocks(a->batch, a->dim, a->groups, lanes);
  Segments sg = scan_segments(a->batch, a->len, a->dim, lanes);
  if (blocks > kMaxBlocks / sg.count) return CR_ERR_UNSUPPORTED;
  sg.E = static_cast<float*>(ws);
  sg.sum = sg.E + (sg.count - 1) * a->batch * a->dim * lanes * kS;
  CR_MODEL_TYPE(a->dt_type, CR_SCAN_LANES(lanes, {
    using TL = Tile<T, G>;
    const size_t bytes = TL::VE * es;
    const bool group_ok = a->groups == 1 || (a->dim / a->groups) % TL::VE == 0;
    ScanOut<T> out;
    out.y = static_cast<T*>(y);
    out.ybs = y_batch_stride;
    out.yts = y_time_stride;
    out.final_state = final_state;
    out.checkpoints = checkpoints;
    out.n_check = cr_selective_scan_checkpoints(a->len);
    out.wide = group_ok && rows_aligned(a->u, a->u_batch_stride, a->u_time_stride, es, bytes) &&
               rows_aligned(a->dt, a->dt_batch_stride, a->dt_time_stride, es, bytes) &&
               (a->z == nullptr ||
                rows_aligned(a->z, a->z_batch_stride, a->z_time_stride, es, bytes));
    out.wide_y = group_ok && rows_aligned(y, y_batch_stride, y_time_stride, es, bytes);
    out.wide_BC = a->dstate % kS == 0 &&
                  rows_aligned(a->B, a->B_batch_stride, a->B_time_stride, es, kS * es) &&
                  rows_aligned(a->C, a->C_batch_stride, a->C_time_stride, es, kS * es);
    if (sg.count > 1)
      CR_LAUNCH(kKSelectiveScanStates, s,
                selective_scan_kernel<T, G, true>
                <<<(unsigned)(blocks * (sg.count - 1)), kScanThreads, 0, s>>>(scan_in<T>(a), out,
                                                                              sg));
    CR_LAUNCH(kKSelectiveScan, s,
              selective_scan_kernel<T, G, false>
              <<<(unsigned)(blocks * sg.count), kScanThreads, 0, s>>>(scan_in<T>(a), out, sg));
  }));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

static int64_t backward_warps(int64_t dim, int32_t groups, int lanes) {
  return cr::ceil_div(dim / groups, cr::kScanThreads / lanes) * (cr::kScanThreads / 32);
}

size_t cr_selective_scan_backward_workspace_bytes(int64_t batch, int64_t len, int64_t dim,
                                                  int32_t dstate, int32_t groups) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || dstate < 1 || groups < 1 || dim % groups != 0) return 0;
  const int lanes = scan_lanes(dstate);
  const size_t bc = (size_t)batch * len * groups * backward_warps(dim, groups, lanes) * 2 *
                    (lanes * kS) * 4;
  return round256(bc) + round256((size_t)batch * dim * (dstate + 2) * 4) + 256;
}

cr_status cr_selective_scan_backward(const cr_selective_scan_args* a,
                                     const cr_selective_scan_grads* g, void* ws,
                                     size_t ws_bytes, void* stream) {
  using namespace cr;
  const cr_status ok = check_scan(a, false);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt_type);
  if (g == nullptr || g->dy_batch_stride < 0 || g->dy_time_stride < 0) return CR_ERR_INVALID_ARG;
  if (a->dim == 0) return CR_OK;
  if (g->dA == nullptr) return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->len > 0 &&
      (g->dy == nullptr || g->checkpoints == nullptr || g->du == nullptr || g->ddt == nullptr ||
       g->dB == nullptr || g->dC == nullptr || (a->z != nullptr && g->dz == nullptr)))
    return CR_ERR_INVALID_ARG;
  const void* ins[6] = {a->u, a->dt, a->z, a->B, a->C, g->dy};
  const void* outs[5] = {g->du, g->ddt, g->dz, g->dB, g->dC};
  for (const void* o : outs) {
    if (!ptr_aligned(o, es)) return CR_ERR_INVALID_ARG;
    for (const void* i : ins)
      if (o != nullptr && o == i) return CR_ERR_INVALID_ARG;
  }
  if (!ptr_aligned(g->dy, es) || !ptr_aligned(g->dfinal, 4) || !ptr_aligned(g->checkpoints, 4) ||
      !ptr_aligned(g->dA, 4) || !ptr_aligned(g->dD, 4) || !ptr_aligned(g->ddt_bias, 4) ||
      !ptr_aligned(g->dstate, 4))
    return CR_ERR_INVALID_ARG;
  const size_t need = cr_selective_scan_backward_workspace_bytes(a->batch, a->len, a->dim,
                                                                 a->dstate, a->groups);
  if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < need) return CR_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int lanes = scan_lanes(a->dstate);
  const int64_t warps = backward_warps(a->dim, a->groups, lanes);
  const int64_t rows = a->batch * a->len * a->groups;
  float* part_BC = static_cast<float*>(ws);
  float* part_A = reinterpret_cast<float*>(
      static_cast<char*>(ws) + round256((size_t)rows * warps * 2 * (lanes * kS) * 4));
  if (a->batch > 0) {
    const unsigned blocks = (unsigned)scan_blocks(a->batch, a->dim, a->groups, lanes);
    const int64_t n_check = cr_selective_scan_checkpoints(a->len);
    CR_MODEL_TYPE(a->dt_type, CR_SCAN_LANES(lanes, {
      ScanBack<T> o;
      o.dy = static_cast<const T*>(g->dy);
      o.dybs = g->dy_batch_stride;
      o.dyts = g->dy_time_stride;
      o.dfinal = g->dfinal;
      o.checkpoints = g->checkpoints;
      o.du = static_cast<T*>(g->du);
      o.ddt = static_cast<T*>(g->ddt);
      o.dz = a->z != nullptr ? static_cast<T*>(g->dz) : nullptr;
      o.dstate = g->dstate;
      o.part_BC = part_BC;
      o.part_A = part_A;
      o.warps = warps;
      CR_LAUNCH(kKSelectiveScanBackward, s,
                selective_scan_backward_kernel<T, G><<<blocks, kScanThreads, 0, s>>>(
                    scan_in<T>(a), o, n_check));
    }));
    if (cudaGetLastError() != cudaSuccess) return CR_ERR_CUDA;
    const int64_t sums = ceil_div(rows * 2 * a->dstate, kScanThreads);
    if (sums > kMaxBlocks) return CR_ERR_UNSUPPORTED;
    if (sums > 0) {
      CR_MODEL_TYPE(a->dt_type, {
        CR_LAUNCH(kKSelectiveScanSum, s,
                  selective_scan_sum_bc_kernel<T><<<(unsigned)sums, kScanThreads, 0, s>>>(
                      part_BC, rows, warps, lanes * kS, a->dstate, static_cast<T*>(g->dB),
                      static_cast<T*>(g->dC)));
      });
    }
  }
  CR_LAUNCH(kKSelectiveScanSum, s,
            selective_scan_sum_a_kernel<<<(unsigned)ceil_div(a->dim * (a->dstate + 2),
                                                             kScanThreads),
                                          kScanThreads, 0, s>>>(
                part_A, a->batch, a->dim, a->dstate, g->dA, g->dD, g->ddt_bias));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

cr_status cr_selective_scan_step(const cr_selective_scan_args* a, float* state,
                                 int64_t state_rows, const void* slots, void* y,
                                 int64_t y_batch_stride, void* stream) {
  using namespace cr;
  const cr_status ok = check_scan(a, true);
  if (ok != CR_OK) return ok;
  const size_t es = model_esize(a->dt_type);
  if (state_rows < 0 || y_batch_stride < 0) return CR_ERR_INVALID_ARG;
  if (slots != nullptr ? !index_width_ok(a->index_bytes) || !ptr_aligned(slots, a->index_bytes)
                       : state_rows < a->batch)
    return CR_ERR_INVALID_ARG;
  if (a->batch == 0 || a->dim == 0) return CR_OK;
  if (y == nullptr || y == a->u || y == a->dt || y == a->z ||
      (state == nullptr && state_rows > 0) || (a->batch > 1 && y_batch_stride < a->dim))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(y, es) || !ptr_aligned(state, 4)) return CR_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int lanes = scan_lanes(a->dstate);
  const unsigned blocks = (unsigned)scan_blocks(a->batch, a->dim, a->groups, lanes);
  CR_MODEL_TYPE(a->dt_type, CR_SCAN_LANES(lanes, {
    CR_LAUNCH(kKSelectiveScanStep, s,
              selective_scan_step_kernel<T, G><<<blocks, kScanThreads, 0, s>>>(
                  scan_in<T>(a), state, state_rows, slots, static_cast<T*>(y), y_batch_stride));
  }));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
