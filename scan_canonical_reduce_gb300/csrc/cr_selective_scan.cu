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
#include <algorithm>
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
template <class T, int V, int NACC, int ALL, int PER_ROW>
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
  __device__ __forceinline__ void load(int left, Raw<T, V> (&out)[NACC][2]) {
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
template <class TL, class T>
__device__ __forceinline__ void tile_put_states(const Raw<T, kS> (&in)[TL::NBC][2], float4* tile) {
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
  bool wide, wide_y, wide_BC, wide_check;
};

#ifndef CR_SCAN_BLOCKS
#define CR_SCAN_BLOCKS 4
#endif
template <class T, int G, bool kStates>
__global__ void __launch_bounds__(kScanThreads, CR_SCAN_BLOCKS)
selective_scan_kernel(ScanIn<T> in, ScanOut<T> out, Segments sg) {
  using TL = Tile<T, G>;
  constexpr int VE = TL::VE;
  __shared__ float4 dd[TL::TP * TL::CH];
  __shared__ float4 Bs[TL::ACC_BC * 2];
  __shared__ float4 Cs[kStates ? 1 : TL::ACC_BC * 2];
  __shared__ __align__(16) float ys[kStates ? 4 : TL::TT * TL::YS];
  __shared__ __align__(16) float Ds[TL::CH], biases[TL::CH];

  const int tid = threadIdx.x, g = Lanes<G>::g(), c = Lanes<G>::c(), n0 = g * kS;
  const int64_t per_group = (in.group_dim + TL::CH - 1) / TL::CH;
  const int64_t segs = kStates ? sg.count - 1 : sg.count;
  int64_t blk, seg, first;
  const int64_t i = divide(blockIdx.x, per_group * in.groups, blk), b = divide(i, segs, seg);
  const int64_t group = divide(blk, per_group, first);
  first *= TL::CH;
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
  F2 A[kS];
  float h[kS] = {0.0f, 0.0f, 0.0f, 0.0f};
  {
    float a[kS];
    load_states(in.A + d * in.N, n0, in.N, a);
#pragma unroll
    for (int k = 0; k < kS; ++k) A[k] = pack2(a[k] * kLog2e, a[k] * kLog2e);
  }
  if (!kStates) {
    if (in.state != nullptr) load_states(in.state + (b * in.dim + d) * in.N, n0, in.N, h);
    const float* E = sg.E + (b * in.dim + d) * TL::NP + n0;
    const float* sum = sg.sum + b * in.dim + d;
#pragma unroll 4
    for (int64_t s = 0; s < seg; ++s) {
      const float4 e4 = *reinterpret_cast<const float4*>(E + s * in.batch * in.dim * TL::NP);
      const float x = sum[s * in.batch * in.dim], e[kS] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        float a, a2;
        unpack2(A[k], a, a2);
        h[k] = fmaf(exp2_fast(x * a), h[k], e[k]);
      }
    }
  }

  using RowsE = Rows<T, VE, TL::NL, TL::ACC, TL::NV>;
  using RowsBC = Rows<T, kS, TL::NBC, TL::ACC_BC, G>;
  static_assert(kScanThreads % TL::NV == 0, "a thread's accesses are of one column");
  RowsE ru(in.u + b * in.ubs + d0, in.uts, begin, TL::TT, channels, out.wide);
  RowsE rd(in.dt + b * in.dbs + d0, in.dts, begin, TL::TT, channels, out.wide);
  RowsE rz(in.z + b * in.zbs + d0, in.zts, begin, TL::TT, channels, out.wide);
  RowsBC rB(in.B + b * in.Bbs + group * in.N, in.Bts, begin, TL::TT, in.N, out.wide_BC);
  RowsBC rC(in.C + b * in.Cbs + group * in.N, in.Cts, begin, TL::TT, in.N, out.wide_BC);
  const bool gated = !kStates && in.z != nullptr;
  Raw<T, VE> pu[TL::NL][2], pd[TL::NL][2], pz[TL::NL][2];
  Raw<T, kS> pB[TL::NBC][2], pC[TL::NBC][2];
  auto load = [&](int left) {
    ru.load(left, pu);
    rd.load(left, pd);
    if (gated) rz.load(left, pz);
    rB.load(left, pB);
    if (!kStates) rC.load(left, pC);
  };
  const int c0 = tid % TL::NV * VE;  // this thread's elements: channels c0 .. c0 + have
  const int have = min(VE, channels - c0);
  T* yp = out.y + b * out.ybs + (begin + tid / TL::NV * 2) * out.yts + d0 + c0;
  load((int)min(stop - begin, (int64_t)TL::TT));
  __syncthreads();  // Ds, biases
  F2 total = 0;

  int64_t t0 = begin;
  for (; t0 < stop; t0 += TL::TT) {
    const int left = (int)min(stop - t0, (int64_t)TL::TT);
    // elements: delta and delta u into the tile; u and z stay for the end
    Raw<T, VE> ku[TL::NL][2], kz[TL::NL][2];
    const Pack<float, VE> bias = *reinterpret_cast<const Pack<float, VE>*>(biases + c0);
#pragma unroll
    for (int i = 0; i < TL::NL; ++i) {
      const int idx = i * kScanThreads + tid, tp = idx / TL::NV;
      const int at = TL::slot(tp, c0) * 16;
      const bool in0 = 2 * tp < left, in1 = 2 * tp + 1 < left;
      float a[VE], a1[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        a[k] = pd[i][0].get(k) + bias.v[k];
        a1[k] = pd[i][1].get(k) + bias.v[k];
      }
      if (in.softplus) {  // all of them in one block: their chains overlap
#pragma unroll
        for (int k = 0; k < VE; ++k) softplus2(a[k], a1[k]);
      }
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        a[k] = in0 ? a[k] : 0.0f;
        a1[k] = in1 ? a1[k] : 0.0f;
        if (TL::ACC % kScanThreads == 0 || idx < TL::ACC)
          *reinterpret_cast<float4*>(reinterpret_cast<char*>(dd) + (at ^ (k * 16))) =
              make_float4(a[k], a1[k], a[k] * pu[i][0].get(k), a1[k] * pu[i][1].get(k));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!kStates) ku[i][j] = pu[i][j];
        if (gated) kz[i][j] = pz[i][j];
      }
    }
    tile_put_states<TL>(pB, Bs);
    if (!kStates) tile_put_states<TL>(pC, Cs);
    __syncthreads();
    if (t0 + TL::TT < stop) load((int)min(stop - t0 - TL::TT, (int64_t)TL::TT));

    // recurrence
    const float4* dl = dd + TL::slot(0, c);
    const float4 *Bl = Bs + 2 * g, *Cl = Cs + 2 * g;
    float* yl = ys + c;
#pragma unroll 1
    for (int tb = 0; tb < TL::TT; tb += kCheckpoint) {
      if (!kStates && out.checkpoints != nullptr && live && t0 + tb < end)
        store_states(out.checkpoints +
                         ((b * out.n_check + (t0 + tb) / kCheckpoint) * in.dim + d) * in.N,
                     n0, in.N, out.wide_check, h);
      // straight code: the reads and decays of later steps run ahead
      float4 e_next, B_next[2], C_next[2];
      auto read = [&](int tp) {
        e_next = dl[tp * TL::CH];
        B_next[0] = Bl[tp * 2 * G], B_next[1] = Bl[tp * 2 * G + 1];
        if (!kStates) C_next[0] = Cl[tp * 2 * G], C_next[1] = Cl[tp * 2 * G + 1];
        else C_next[0] = C_next[1] = B_next[0];
      };
      read(0);
      F2 q[2] = {0, 0};
      auto finish = [&](int t4) {
        float v[4];
        sum_lanes4<G>(q[0], q[1], g, v);
        float* y = yl + t4 * 4 * TL::YS;
        if (G == 1) {
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k * TL::YS] = v[k];
        } else if (G == 2) {
#pragma unroll
          for (int k = 0; k < 2; ++k) y[(2 * g + k) * TL::YS] = v[k];
        } else if (G == 4 || g < 4) {
          y[(2 * (g & 1) + (g >> 1 & 1)) * TL::YS] = v[0];
        }
      };
#pragma unroll
      for (int t4 = 0; t4 < kCheckpoint / 4; ++t4) {
        F2 p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 e = e_next, B[2] = {B_next[0], B_next[1]};
          const float4 C[2] = {C_next[0], C_next[1]};
          if (2 * t4 + j + 1 < kCheckpoint / 2) read(2 * t4 + j + 1);
          if (kStates) total = add2(total, pack2(e.x, e.y));
          p[j] = lane_steps<!kStates>(A, h, e, B, C);
        }
        if (!kStates) {
          if (t4 > 0) finish(t4 - 1);
          q[0] = p[0];
          q[1] = p[1];
        }
      }
      if (!kStates) finish(kCheckpoint / 4 - 1);
      dl += kCheckpoint / 2 * TL::CH;
      Bl += kCheckpoint * G;
      if (!kStates) Cl += kCheckpoint * G;
      yl += kCheckpoint * TL::YS;
    }
    __syncthreads();

    // elements: D u, the gate, and out
    if (!kStates) {
      const Pack<float, VE> Dv = *reinterpret_cast<const Pack<float, VE>*>(Ds + c0);
      const int rows = (int)min(end - t0, (int64_t)TL::TT);
#pragma unroll
      for (int i = 0; i < TL::NL; ++i) {
        const int idx = i * kScanThreads + tid, tp = idx / TL::NV;
        if (TL::ACC % kScanThreads != 0 && idx >= TL::ACC) continue;
        float f[2][VE];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const Pack<float, VE> yv =
              *reinterpret_cast<const Pack<float, VE>*>(ys + (2 * tp + j) * TL::YS + c0);
#pragma unroll
          for (int k = 0; k < VE; ++k) f[j][k] = fmaf(Dv.v[k], ku[i][j].get(k), yv.v[k]);
        }
        if (gated) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < VE; ++k) {
              const float z = kz[i][j].get(k);
              f[j][k] *= z * sigmoid(z);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = 2 * tp + j;
          if (t >= left) {
#pragma unroll
            for (int k = 0; k < VE; ++k) f[j][k] = 0.0f;
          }
          if (t < rows && have > 0)
            store_f32<T, VE>(yp + (i * (kScanThreads / TL::NV) * 2 + j) * out.yts,
                             out.wide_y && have == VE, have, f[j]);
        }
      }
      yp += TL::TT * out.yts;
    }
  }
  if constexpr (kStates) {
    if (live) {
      const int64_t row = (seg * in.batch + b) * in.dim + d;
      *reinterpret_cast<float4*>(sg.E + row * TL::NP + n0) = make_float4(h[0], h[1], h[2], h[3]);
      float lo, hi;
      unpack2(total, lo, hi);
      if (g == 0) sg.sum[row] = lo + hi;
    }
  } else {
  for (int64_t t = t0; t < end; ++t)  // past the sequence's length
    for (int k = tid; k < channels; k += kScanThreads)
      out.y[b * out.ybs + t * out.yts + d0 + k] = from_f32<T>(0.0f);
  if (out.final_state != nullptr && seg == sg.count - 1 && live) {
#pragma unroll
    for (int k = 0; k < kS; ++k)
      if (n0 + k < in.N) out.final_state[(b * in.dim + d) * in.N + n0 + k] = h[k];
  }
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
  float* part_BC;  // [batch][len][groups][blocks][2][NP]: dB, dC
  float* part_A;   // [batch][dim][N + 2]: dA, dD, ddt_bias
  int64_t n_check;
  bool wide, wide_out, wide_BC, wide_check;
};

// Sums over the channels of a warp. A lane holds, for a pair of steps, dB
// (v[0..3]) and dC (v[4..7]) of its four state slots; slot k of lane c is
// state k ^ 2 where c is in the upper half of the warp's channels, so that
// the first level keeps slots 0 and 1 and sends 2 and 3 in every lane. The
// next levels halve over slots, kind and step; at the end lane c owns what
// its bits say (see owned()).
template <int G>
struct ChannelSum {
  static constexpr int L = 32 / G;  // lanes that are summed
  static constexpr int kPairs = L >= 8 ? 1 : L == 4 ? 2 : L == 2 ? 4 : 8;  // left of 8

  static __device__ __forceinline__ F2 exchange(F2 keep, F2 send, int mask) {
    float a, b;
    unpack2(send, a, b);
    a = __shfl_xor_sync(~0u, a, mask);
    b = __shfl_xor_sync(~0u, b, mask);
    return add2(keep, pack2(a, b));
  }
  static __device__ __forceinline__ F2 select(bool s, F2 a, F2 b) { return s ? a : b; }

  // v[8] -> v[0 .. kPairs)
  static __device__ __forceinline__ void run(F2 (&v)[8], int c) {
    if (L >= 2) {  // slots {0, 1} or {2, 3}: v = B0 B1 C0 C1
      v[0] = exchange(v[0], v[2], L / 2);
      v[1] = exchange(v[1], v[3], L / 2);
      v[2] = exchange(v[4], v[6], L / 2);
      v[3] = exchange(v[5], v[7], L / 2);
    }
    if (L >= 4) {  // slot 0 or 1: v = B C
      const bool up = c & (L / 4);
      const F2 b = exchange(select(up, v[1], v[0]), select(up, v[0], v[1]), L / 4);
      v[1] = exchange(select(up, v[3], v[2]), select(up, v[2], v[3]), L / 4);
      v[0] = b;
    }
    if (L >= 8) {  // B or C
      const bool up = c & (L / 8);
      v[0] = exchange(select(up, v[1], v[0]), select(up, v[0], v[1]), L / 8);
    }
#pragma unroll
    for (int s = L / 16; s >= 1; s /= 2) v[0] = exchange(v[0], v[0], s);
  }
  // Which (kind, slot) pair i of lane c is: kind * NP + state, within a row.
  static __device__ __forceinline__ int owned(int i, int c, int g) {
    constexpr int NP = G * kS;
    int kind = i / (kPairs == 8 ? 4 : kPairs == 4 ? 2 : 1) % 2, slot = i % (kPairs == 8 ? 4 : 2);
    if (L == 2) slot = i % 2 + (c & 1 ? 2 : 0);
    if (L >= 4) slot = (c & (L / 2) ? 2 : 0) + (c & (L / 4) ? 1 : 0);
    if (L >= 8) kind = c & (L / 8) ? 1 : 0;
    return kind * NP + g * kS + slot;
  }
  // Lanes that only repeat another's result (L > 8) do not write.
  static __device__ __forceinline__ bool writes(int c) { return L <= 8 || c % (L > 8 ? L / 8 : 1) == 0; }
};

// A block walks its channels' tiles of kCheckpoint steps from the last to the
// first: it takes the tile's states forward from the checkpoint, holding all
// of them in registers, then the adjoint states back, with the decays
// computed again (holding them too spilled registers).
#ifndef CR_SCAN_BACK_BLOCKS
#define CR_SCAN_BACK_BLOCKS 2
#endif
template <class T, int G>
__global__ void __launch_bounds__(kScanThreads, CR_SCAN_BACK_BLOCKS)
selective_scan_backward_kernel(ScanIn<T> in, ScanBack<T> o) {
  using TL = Tile<T, G, kCheckpoint>;
  using CS = ChannelSum<G>;
  constexpr int VE = TL::VE, TT = TL::TT, TP = TL::TP, NP = TL::NP, kWarps = kScanThreads / 32;
  __shared__ float4 dd[TP * TL::CH];               // delta, delta', du, du'
  __shared__ __align__(16) float2 pp[TP * TL::CH];  // p, p'
  __shared__ float4 Bs[TL::ACC_BC * 2], Cs[TL::ACC_BC * 2];
  // y, sum_n g B, sum_n q A of the steps
  __shared__ __align__(16) float ys[TT * TL::YS], gs[TT * TL::YS], qs[TT * TL::YS];
  __shared__ float2 sums[kWarps * TP * 2 * NP];
  __shared__ __align__(16) float Ds[TL::CH], biases[TL::CH];

  const int tid = threadIdx.x, g = Lanes<G>::g(), c = Lanes<G>::c(), n0 = g * kS;
  const int lane_c = c % CS::L;
  const int flip = (CS::L >= 2 && (lane_c & (CS::L / 2))) ? 2 : 0;  // slot k holds state k ^ flip
  const int64_t per_group = (in.group_dim + TL::CH - 1) / TL::CH;
  int64_t blk, block;
  const int64_t b = divide(blockIdx.x, per_group * in.groups, blk);
  const int64_t group = divide(blk, per_group, block), first = block * TL::CH;
  const int channels = (int)min((int64_t)TL::CH, in.group_dim - first);
  const int64_t d0 = group * in.group_dim + first;
  const bool live = c < channels;
  const int64_t d = d0 + (live ? c : 0);
  const int64_t len = sequence_length(in.lengths, in.index_bytes, b, in.len);
  const int64_t row = (b * in.dim + d) * in.N;

  if (tid < TL::CH) {
    Ds[tid] = (in.D != nullptr && tid < channels) ? in.D[d0 + tid] : 0.0f;
    biases[tid] = (in.dt_bias != nullptr && tid < channels) ? in.dt_bias[d0 + tid] : 0.0f;
  }
  F2 A[kS], dA[kS];
  float carry[kS] = {0.0f, 0.0f, 0.0f, 0.0f};
  {
    float a[kS], f[kS] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_states(in.A + d * in.N, n0, in.N, a);
    if (o.dfinal != nullptr && live) load_states(o.dfinal + row, n0, in.N, f);
#pragma unroll
    for (int k = 0; k < kS; ++k) {
      A[k] = pack2(flip ? a[k ^ 2] : a[k], flip ? a[k ^ 2] : a[k]);
      carry[k] = flip ? f[k ^ 2] : f[k];
      dA[k] = 0;
    }
  }

  // Tiles past the sequence's length: zeros.
  const int64_t tiles = (len + TT - 1) / TT;
  const int c0 = tid % TL::NV * VE, have = min(VE, channels - c0);
  for (int64_t t = tiles * TT; t < in.len; ++t) {
    for (int k = tid; k < channels; k += kScanThreads) {
      const int64_t at = (b * in.len + t) * in.dim + d0 + k;
      o.du[at] = o.ddt[at] = from_f32<T>(0.0f);
      if (o.dz != nullptr) o.dz[at] = from_f32<T>(0.0f);
    }
    for (int k = tid; k < 2 * NP; k += kScanThreads)
      o.part_BC[((b * in.len + t) * in.groups * per_group + blk) * 2 * NP + k] = 0.0f;
  }

  using RowsE = Rows<T, VE, TL::NL, TL::ACC, TL::NV>;
  using RowsBC = Rows<T, kS, TL::NBC, TL::ACC_BC, G>;
  const int64_t last = (tiles - 1) * TT;
  RowsE ru(in.u + b * in.ubs + d0, in.uts, last, -TT, channels, o.wide);
  RowsE rd(in.dt + b * in.dbs + d0, in.dts, last, -TT, channels, o.wide);
  RowsE rz(in.z + b * in.zbs + d0, in.zts, last, -TT, channels, o.wide);
  RowsE ry(o.dy + b * o.dybs + d0, o.dyts, last, -TT, channels, o.wide);
  RowsBC rB(in.B + b * in.Bbs + group * in.N, in.Bts, last, -TT, in.N, o.wide_BC);
  RowsBC rC(in.C + b * in.Cbs + group * in.N, in.Cts, last, -TT, in.N, o.wide_BC);
  const bool gated = in.z != nullptr;
  Raw<T, VE> pu[TL::NL][2], pd[TL::NL][2], pz[TL::NL][2], py[TL::NL][2];
  Raw<T, kS> pB[TL::NBC][2], pC[TL::NBC][2];
  float next[kS];
  auto load = [&](int64_t tile) {
    const int left = (int)min(len - tile * TT, (int64_t)TT);
    ru.load(left, pu);
    rd.load(left, pd);
    if (gated) rz.load(left, pz);
    ry.load(left, py);
    rB.load(left, pB);
    rC.load(left, pC);
    const float* q = o.checkpoints + ((b * o.n_check + tile) * in.dim + d) * in.N;
    read_states(q, n0, in.N, o.wide_check, next);
  };
  if (tiles > 0) load(tiles - 1);
  __syncthreads();  // Ds, biases
  float dD[VE], dbias[VE];
#pragma unroll
  for (int k = 0; k < VE; ++k) dD[k] = dbias[k] = 0.0f;

  for (int64_t tile = tiles - 1; tile >= 0; --tile) {
    const int64_t t0 = tile * TT;
    const int left = (int)min(len - t0, (int64_t)TT);
    // elements: delta, delta u and p into the tile
    Raw<T, VE> ku[TL::NL][2], kd[TL::NL][2], kz[TL::NL][2], ky[TL::NL][2];
    const Pack<float, VE> bias = *reinterpret_cast<const Pack<float, VE>*>(biases + c0);
    const Pack<float, VE> Dv = *reinterpret_cast<const Pack<float, VE>*>(Ds + c0);
#pragma unroll
    for (int i = 0; i < TL::NL; ++i) {
      const int idx = i * kScanThreads + tid, tp = idx / TL::NV;
      const int at = TL::slot(tp, c0);
      const bool in0 = 2 * tp < left, in1 = 2 * tp + 1 < left;
      float a[VE], a1[VE], p[VE], p1[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        a[k] = pd[i][0].get(k) + bias.v[k];
        a1[k] = pd[i][1].get(k) + bias.v[k];
        p[k] = py[i][0].get(k);
        p1[k] = py[i][1].get(k);
      }
      if (in.softplus) {
#pragma unroll
        for (int k = 0; k < VE; ++k) softplus2(a[k], a1[k]);
      }
      if (gated) {
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float z = pz[i][0].get(k), z1 = pz[i][1].get(k);
          p[k] *= z * sigmoid(z);
          p1[k] *= z1 * sigmoid(z1);
        }
      }
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        a[k] = in0 ? a[k] : 0.0f;
        a1[k] = in1 ? a1[k] : 0.0f;
        if (TL::ACC % kScanThreads == 0 || idx < TL::ACC) {
          dd[at ^ k] = make_float4(a[k], a1[k], a[k] * pu[i][0].get(k), a1[k] * pu[i][1].get(k));
          pp[at ^ k] = make_float2(p[k], p1[k]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ku[i][j] = pu[i][j];
        kd[i][j] = pd[i][j];
        ky[i][j] = py[i][j];
        if (gated) kz[i][j] = pz[i][j];
      }
    }
    tile_put_states<TL>(pB, Bs);
    tile_put_states<TL>(pC, Cs);
    float h[TT + 1][kS];
#pragma unroll
    for (int k = 0; k < kS; ++k) h[0][k] = flip ? next[k ^ 2] : next[k];
    __syncthreads();
    if (tile > 0) load(tile - 1);

    // the states, forward; the quads of B and C in slot order
    const float4* dl = dd + TL::slot(0, c);
    const float2* pl = pp + TL::slot(0, c);
    const float4 *Bl = Bs + 2 * g, *Cl = Cs + 2 * g;
    const int q0 = flip / 2, q1 = 1 - q0;
    F2 yq[2] = {0, 0};  // of the four steps before: summed behind the next ones
    auto put_y = [&](int t4) {
      float v[4];
      sum_lanes4<G>(yq[0], yq[1], g, v);
      float* y = ys + t4 * 4 * TL::YS + c;
      if (G == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k * TL::YS] = v[k];
      } else if (G == 2) {
#pragma unroll
        for (int k = 0; k < 2; ++k) y[(2 * g + k) * TL::YS] = v[k];
      } else if (G == 4 || g < 4) {
        y[(2 * (g & 1) + (g >> 1 & 1)) * TL::YS] = v[0];
      }
    };
#pragma unroll
    for (int t4 = 0; t4 < TT / 4; ++t4) {
      F2 yp[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int tp = t4 * 2 + j, t = tp * 2;
        const float4 e = dl[tp * TL::CH];
        const F2 delta = pack2(e.x * kLog2e, e.y * kLog2e), du = pack2(e.z, e.w);
        const float4 B[2] = {Bl[tp * 2 * G + q0], Bl[tp * 2 * G + q1]};
        const float4 C[2] = {Cl[tp * 2 * G + q0], Cl[tp * 2 * G + q1]};
#pragma unroll
        for (int k = 0; k < kS; ++k) {
          const F2 Bk = k % 2 ? pack2(B[k / 2].z, B[k / 2].w) : pack2(B[k / 2].x, B[k / 2].y);
          const F2 Ck = k % 2 ? pack2(C[k / 2].z, C[k / 2].w) : pack2(C[k / 2].x, C[k / 2].y);
          float x0, x1, b0, b1;
          unpack2(mul2(delta, A[k]), x0, x1);
          unpack2(mul2(du, Bk), b0, b1);
          h[t + 1][k] = fmaf(exp2_fast(x0), h[t][k], b0);
          h[t + 2][k] = fmaf(exp2_fast(x1), h[t + 1][k], b1);
          const F2 hp = pack2(h[t + 1][k], h[t + 2][k]);
          yp[j] = k == 0 ? mul2(Ck, hp) : fma2(Ck, hp, yp[j]);
        }
      }
      if (t4 > 0) put_y(t4 - 1);
      yq[0] = yp[0];
      yq[1] = yp[1];
    }
    put_y(TT / 4 - 1);

    // the adjoint states, backward; the tile is read again, so that nothing of
    // the pass above but h is held in registers
    asm volatile("" ::: "memory");
    // the sums of a pair of steps: their exchanges are issued after the next
    // pair's arithmetic, which hides them
    F2 pv[8], pg = 0, pq = 0;
    auto finish = [&](int tp) {
      const int t = tp * 2;
      CS::run(pv, lane_c);
      if (CS::writes(lane_c)) {
#pragma unroll
        for (int i = 0; i < CS::kPairs; ++i) {
          float lo, hi;
          unpack2(pv[i], lo, hi);
          sums[(tid / 32 * TP + tp) * 2 * NP + CS::owned(i, lane_c, g)] = make_float2(lo, hi);
        }
      }
      float w[4];
      sum_lanes4<G>(pg, pq, g, w);
      float *gl = gs + t * TL::YS + c, *ql = qs + t * TL::YS + c;
      if (G == 1) {
        gl[0] = w[0], gl[TL::YS] = w[1], ql[0] = w[2], ql[TL::YS] = w[3];
      } else if (G == 2) {
        float* q = g ? ql : gl;
        q[0] = w[0], q[TL::YS] = w[1];
      } else if (G == 4 || g < 4) {
        (g & 1 ? ql : gl)[(g >> 1 & 1) * TL::YS] = w[0];
      }
    };
#pragma unroll
    for (int tp = TP - 1; tp >= 0; --tp) {
      const int t = tp * 2;
      const float4 e = dl[tp * TL::CH];
      const float2 p2 = pl[tp * TL::CH];
      const F2 delta = pack2(e.x, e.y), du = pack2(e.z, e.w), p = pack2(p2.x, p2.y);
      const F2 delta2 = pack2(e.x * kLog2e, e.y * kLog2e);
      const float4 B[2] = {Bl[tp * 2 * G + q0], Bl[tp * 2 * G + q1]};
      const float4 C[2] = {Cl[tp * 2 * G + q0], Cl[tp * 2 * G + q1]};
      F2 v[8], gB = 0, qA = 0;
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        const F2 Bk = k % 2 ? pack2(B[k / 2].z, B[k / 2].w) : pack2(B[k / 2].x, B[k / 2].y);
        const F2 Ck = k % 2 ? pack2(C[k / 2].z, C[k / 2].w) : pack2(C[k / 2].x, C[k / 2].y);
        float c0, c1, x0, x1;
        unpack2(mul2(Ck, p), c0, c1);
        unpack2(mul2(delta2, A[k]), x0, x1);
        const float g1 = c1 + carry[k], r1 = g1 * exp2_fast(x1);
        const float g0 = c0 + r1, r0 = g0 * exp2_fast(x0);
        carry[k] = r0;
        const F2 gp = pack2(g0, g1), q = pack2(r0 * h[t][k], r1 * h[t + 1][k]);
        dA[k] = fma2(q, delta, dA[k]);
        qA = k == 0 ? mul2(q, A[k]) : fma2(q, A[k], qA);
        gB = k == 0 ? mul2(gp, Bk) : fma2(gp, Bk, gB);
        v[k] = mul2(gp, du);
        v[4 + k] = mul2(p, pack2(h[t + 1][k], h[t + 2][k]));
      }
      if (tp < TP - 1) finish(tp + 1);
#pragma unroll
      for (int k = 0; k < 8; ++k) pv[k] = v[k];
      pg = gB;
      pq = qA;
    }
    finish(0);
    __syncthreads();

    // dB and dC of the block's channels: the warps in order
    for (int k = tid; k < TP * 2 * NP; k += kScanThreads) {
      float2 s = sums[k];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float2 v = sums[w * TP * 2 * NP + k];
        s.x += v.x;
        s.y += v.y;
      }
      const int64_t t = t0 + k / (2 * NP) * 2;
      const int64_t stride = (int64_t)in.groups * per_group * 2 * NP;
      float* q = o.part_BC + (b * in.len + t) * stride +
                 blk * 2 * NP + k % (2 * NP);
      if (t < in.len) q[0] = s.x;
      if (t + 1 < in.len) q[stride] = s.y;
    }
    // elements: du, ddt, dz out
#pragma unroll
    for (int i = 0; i < TL::NL; ++i) {
      const int idx = i * kScanThreads + tid, tp = idx / TL::NV;
      if (TL::ACC % kScanThreads != 0 && idx >= TL::ACC) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 2 * tp + j;
        const Pack<float, VE> yv = *reinterpret_cast<const Pack<float, VE>*>(ys + t * TL::YS + c0);
        const Pack<float, VE> gv = *reinterpret_cast<const Pack<float, VE>*>(gs + t * TL::YS + c0);
        const Pack<float, VE> qv = *reinterpret_cast<const Pack<float, VE>*>(qs + t * TL::YS + c0);
        float fu[VE], fd[VE], fz[VE], p[VE], u[VE];
        const bool in_seq = t < left;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          u[k] = ku[i][j].get(k);
          const float4 e = dd[TL::slot(tp, c0) ^ k];
          const float2 p2 = pp[TL::slot(tp, c0) ^ k];
          p[k] = j ? p2.y : p2.x;
          fu[k] = fmaf(j ? e.y : e.x, gv.v[k], Dv.v[k] * p[k]);
          fd[k] = fmaf(u[k], gv.v[k], qv.v[k]);
          fz[k] = 0.0f;
        }
        if (in.softplus) {
#pragma unroll
          for (int k = 0; k < VE; ++k) fd[k] *= sigmoid(kd[i][j].get(k) + bias.v[k]);
        }
        if (gated) {
#pragma unroll
          for (int k = 0; k < VE; ++k) {
            const float z = kz[i][j].get(k), sg = sigmoid(z);
            fz[k] = ky[i][j].get(k) * fmaf(Dv.v[k], u[k], yv.v[k]) * (sg * fmaf(z, 1.0f - sg, 1.0f));
          }
        }
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          if (in_seq) {
            dD[k] = fmaf(p[k], u[k], dD[k]);
            dbias[k] += fd[k];
          } else {
            fu[k] = fd[k] = fz[k] = 0.0f;
          }
        }
        if (t0 + t < in.len && have > 0) {
          const int64_t at = (b * in.len + t0 + t) * in.dim + d0 + c0;
          const bool w = o.wide_out && have == VE;
          store_f32<T, VE>(o.du + at, w, have, fu);
          store_f32<T, VE>(o.ddt + at, w, have, fd);
          if (o.dz != nullptr) store_f32<T, VE>(o.dz + at, w, have, fz);
        }
      }
    }
    // the next tile's elements overwrite dd and pp where this thread read them
  }

  // dD and ddt_bias: the threads of a channel in order
  float* red = ys;  // [rows of threads][CH]
  constexpr int kRows = kScanThreads / TL::NV;
  static_assert(kRows * TL::CH <= TT * TL::YS, "the y tile holds a value of every thread's");
  __syncthreads();
  if (live) {
    float* q = o.part_A + (b * in.dim + d) * (in.N + 2);
#pragma unroll
    for (int k = 0; k < kS; ++k) {
      const int n = n0 + (k ^ flip);
      float lo, hi;
      unpack2(dA[k], lo, hi);
      if (n < in.N) {
        q[n] = lo + hi;
        if (o.dstate != nullptr) o.dstate[row + n] = carry[k];
      }
    }
  }
  for (int pass = 0; pass < 2; ++pass) {
    if (tid / TL::NV < kRows && c0 < TL::CH) {
#pragma unroll
      for (int k = 0; k < VE; ++k) red[tid / TL::NV * TL::CH + c0 + k] = pass ? dbias[k] : dD[k];
    }
    __syncthreads();
    if (tid < channels) {
      float s = 0.0f;
      for (int r = 0; r < kRows; ++r) s += red[r * TL::CH + tid];
      o.part_A[(b * in.dim + d0 + tid) * (in.N + 2) + in.N + pass] = s;
    }
    __syncthreads();
  }
}

// dB and dC: the blocks' partials of a (sequence, step, group), in order.
template <class T>
__global__ void __launch_bounds__(kScanThreads)
selective_scan_sum_bc_kernel(const float* __restrict__ part, int64_t rows, int64_t blocks, int NP,
                             int N, T* __restrict__ dB, T* __restrict__ dC) {
  const int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= rows * 2 * N) return;
  int64_t j;
  const int64_t r = divide(i, 2 * N, j);
  const int which = j >= N, n = (int)j - which * N;
  const float* q = part + r * blocks * 2 * NP + which * NP + n;
  float s = 0.0f;
#pragma unroll 16
  for (int64_t w = 0; w < blocks; ++w) s += q[w * 2 * NP];
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
  int64_t k;
  const int64_t d = divide(i, N + 2, k);
  if (k < N) dA[d * N + k] = s;
  else if (k == N && dD != nullptr) dD[d] = s;
  else if (k == N + 1 && dbias != nullptr) dbias[d] = s;
}

// One token. A warp takes 32 channels of a group: first a lane each, for
// delta, delta u and the gate, then G rounds of 32 / G channels by G lanes
// each, lane = c G + g, so that a round's states are consecutive in memory.
// All rounds' reads are in flight together. kWide: rows of states, A, B and C
// allow accesses of four elements.
template <class T, int G, bool kWide>
__global__ void __launch_bounds__(kScanThreads)
selective_scan_step_kernel(ScanIn<T> in, float* __restrict__ state, int64_t state_rows,
                           const void* __restrict__ slots, T* __restrict__ y, int64_t ybs) {
  constexpr int L = 32 / G, kWarps = kScanThreads / 32;
  constexpr int kAhead = G < 8 ? G : 8;  // rounds in flight
  const int lane = threadIdx.x % 32, g = lane % G;
  const uint32_t warp = blockIdx.x * kWarps + threadIdx.x / 32;
  const uint32_t per_group = (uint32_t)((in.group_dim + 31) / 32);
  const int64_t group = in.groups == 1 ? 0 : warp / per_group;
  const int64_t first = (int64_t)(warp - (uint32_t)group * per_group) * 32;  // in the group
  // the grid's other axes count streams: what depends on them alone is
  // computed once a warp
  const int64_t b = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
  if (b >= in.batch || group >= in.groups || first >= in.group_dim) return;
  const int channels = (int)min((int64_t)32, in.group_dim - first);
  const int64_t d0 = group * in.group_dim + first, d = d0 + min(lane, channels - 1);
  const int64_t slot = slots != nullptr ? load_index(slots, in.index_bytes, b) : b;
  if (slot < 0 || slot >= state_rows) {  // the same for the whole warp
    if (lane < channels) y[b * ybs + d] = from_f32<T>(0.0f);
    return;
  }
  const int n0 = g * kS, have = kWide ? (n0 < in.N ? kS : 0) : min(kS, in.N - n0);
  auto floats = [&](const float* q, bool read, float (&f)[kS]) {
    if (kWide) {
      const float4 v =
          read && have > 0 ? *reinterpret_cast<const float4*>(q) : make_float4(0, 0, 0, 0);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < kS; ++k) f[k] = read && k < have ? q[k] : 0.0f;
    }
  };
  auto elements = [&](const T* q, Raw<T, kS>& r) {
    if (!kWide) r.load(q, false, have);
    else if (have > 0) r.load(q, true, kS);
    else r.zero();
  };
  float* st = state + (slot * in.dim + d0) * in.N + n0;
  const float* A0 = in.A + d0 * in.N + n0;
  float h[kAhead][kS], A[kAhead][kS];
  auto read = [&](int r0) {
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      const int c = (r0 + r) * L + lane / G;
      floats(st + c * in.N, c < channels, h[r]);
      floats(A0 + c * in.N, c < channels, A[r]);
    }
  };
  read(0);
  Raw<T, kS> Braw, Craw;
  elements(in.B + b * in.Bbs + group * in.N + n0, Braw);
  elements(in.C + b * in.Cbs + group * in.N + n0, Craw);
  const float u = to_f32(in.u[b * in.ubs + d]);
  float delta = to_f32(in.dt[b * in.dbs + d]);
  const float z = in.z != nullptr ? to_f32(in.z[b * in.zbs + d]) : 0.0f;
  const float D = in.D != nullptr ? in.D[d] : 0.0f;
  if (in.dt_bias != nullptr) delta += in.dt_bias[d];
  if (in.softplus) delta = softplus(delta);
  const float du = delta * u;
  float B[kS], C[kS], mine = 0.0f;
#pragma unroll
  for (int k = 0; k < kS; ++k) {
    B[k] = Braw.get(k);
    C[k] = Craw.get(k);
  }
#pragma unroll
  for (int r0 = 0; r0 < G; r0 += kAhead) {
    if (r0 > 0) read(r0);
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      const int c = (r0 + r) * L + lane / G;
      const float dc = __shfl_sync(~0u, delta, c), duc = __shfl_sync(~0u, du, c);
      float acc = 0.0f;
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        h[r][k] = fmaf(exp2_fast(dc * (A[r][k] * kLog2e)), h[r][k], duc * B[k]);
        acc = k == 0 ? C[k] * h[r][k] : fmaf(C[k], h[r][k], acc);
      }
      if (c < channels) {
        if (kWide) {
          if (have > 0)
            *reinterpret_cast<float4*>(st + c * in.N) =
                make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
        } else {
#pragma unroll
          for (int k = 0; k < kS; ++k)
            if (k < have) st[c * in.N + k] = h[r][k];
        }
      }
      // back to the lane that has the channel
      const float v = __shfl_sync(~0u, sum_lanes<G>(acc), lane % L * G);
      if (lane / L == r0 + r) mine = v;
    }
  }
  float o = fmaf(D, u, mine);
  if (in.z != nullptr) o *= z * sigmoid(z);
  if (lane < channels) y[b * ybs + d] = from_f32<T>(o);
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
#ifndef CR_SCAN_LEAST
#define CR_SCAN_LEAST 1
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
  if (warps < CR_SCAN_SPLIT_BELOW && warps > 0 && len >= 2 * CR_SCAN_LEAST * kTile) {
    sg.count = CR_SCAN_WARPS / warps;
    const int64_t most = len / (CR_SCAN_LEAST * kTile);
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
  return round256((size_t)(segs - 1) * batch * dim * (scan_lanes(dstate) * kS + 1) * 4) +
         kStatusBytes;
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
  sg.E = reinterpret_cast<float*>(past_status(ws));
  sg.sum = sg.E + (sg.count - 1) * a->batch * a->dim * lanes * kS;
  CR_MODEL_TYPE(a->dt_type, CR_SCAN_LANES(lanes, {
    using TL = Tile<T, G>;
    const size_t bytes = TL::VE * es;  // of an access
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
    out.wide_check = a->dstate % kS == 0 && ptr_aligned(checkpoints, 16);
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

// Blocks that share a group of a sequence: each leaves its own dB and dC.
static int64_t group_blocks(int64_t dim, int32_t groups, int lanes) {
  return cr::ceil_div(dim / groups, cr::kScanThreads / lanes);
}

size_t cr_selective_scan_backward_workspace_bytes(int64_t batch, int64_t len, int64_t dim,
                                                  int32_t dstate, int32_t groups) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || dstate < 1 || groups < 1 || dim % groups != 0) return 0;
  const int lanes = scan_lanes(dstate);
  const size_t bc = (size_t)batch * len * groups * group_blocks(dim, groups, lanes) * 2 *
                    (lanes * kS) * 4;
  return round256(bc) + round256((size_t)batch * dim * (dstate + 2) * 4) + kStatusBytes;
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
  const int64_t parts = group_blocks(a->dim, a->groups, lanes);
  const int64_t rows = a->batch * a->len * a->groups;
  float* part_BC = reinterpret_cast<float*>(past_status(ws));
  float* part_A = reinterpret_cast<float*>(
      past_status(ws) + round256((size_t)rows * parts * 2 * (lanes * kS) * 4));
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
      o.n_check = n_check;
      using TL = Tile<T, G, kCheckpoint>;
      const size_t bytes = TL::VE * es;  // of an access
      const bool group_ok = a->groups == 1 || (a->dim / a->groups) % TL::VE == 0;
      o.wide = group_ok && rows_aligned(a->u, a->u_batch_stride, a->u_time_stride, es, bytes) &&
               rows_aligned(a->dt, a->dt_batch_stride, a->dt_time_stride, es, bytes) &&
               rows_aligned(g->dy, g->dy_batch_stride, g->dy_time_stride, es, bytes) &&
               (a->z == nullptr ||
                rows_aligned(a->z, a->z_batch_stride, a->z_time_stride, es, bytes));
      o.wide_out = group_ok && rows_aligned(g->du, a->dim, a->dim, es, bytes) &&
                   rows_aligned(g->ddt, a->dim, a->dim, es, bytes) &&
                   rows_aligned(o.dz, a->dim, a->dim, es, bytes);
      o.wide_BC = a->dstate % kS == 0 &&
                  rows_aligned(a->B, a->B_batch_stride, a->B_time_stride, es, kS * es) &&
                  rows_aligned(a->C, a->C_batch_stride, a->C_time_stride, es, kS * es);
      o.wide_check = a->dstate % kS == 0 && ptr_aligned(g->checkpoints, 16);
      CR_LAUNCH(kKSelectiveScanBackward, s,
                selective_scan_backward_kernel<T, G><<<blocks, kScanThreads, 0, s>>>(
                    scan_in<T>(a), o));
    }));
    if (cudaGetLastError() != cudaSuccess) return CR_ERR_CUDA;
    const int64_t sums = ceil_div(rows * 2 * a->dstate, kScanThreads);
    if (sums > kMaxBlocks) return CR_ERR_UNSUPPORTED;
    if (sums > 0) {
      CR_MODEL_TYPE(a->dt_type, {
        CR_LAUNCH(kKSelectiveScanSum, s,
                  selective_scan_sum_bc_kernel<T><<<(unsigned)sums, kScanThreads, 0, s>>>(
                      part_BC, rows, parts, lanes * kS, a->dstate, static_cast<T*>(g->dB),
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
  const bool wide = a->dstate % kS == 0 && ptr_aligned(state, 16) && ptr_aligned(a->A, 16) &&
                    rows_aligned(a->B, a->B_batch_stride, 0, es, kS * es) &&
                    rows_aligned(a->C, a->C_batch_stride, 0, es, kS * es);
  constexpr int64_t kRows = 65535;  // of a grid's second and third axes
  const int64_t blocks = ceil_div(ceil_div(a->dim / a->groups, 32) * a->groups, kScanThreads / 32);
  if (ceil_div(a->batch, kRows) > kRows || blocks > kMaxBlocks / 4) return CR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks, (unsigned)std::min(a->batch, kRows),
                  (unsigned)ceil_div(a->batch, kRows));
  CR_MODEL_TYPE(a->dt_type, CR_SCAN_LANES(lanes, {
    auto kernel = wide ? selective_scan_step_kernel<T, G, true>
                       : selective_scan_step_kernel<T, G, false>;
    CR_LAUNCH(kKSelectiveScanStep, s,
              kernel<<<grid, kScanThreads, 0, s>>>(scan_in<T>(a), state, state_rows, slots,
                                                   static_cast<T*>(y), y_batch_stride));
  }));
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
