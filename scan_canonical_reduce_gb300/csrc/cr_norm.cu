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

// (len 0: one batch, whose rows need no division)
__device__ __forceinline__ int64_t row_offset(int64_t r, int64_t len, Rows2 s) {
  if (len == 0) return r * s.ts;
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
// From the sums of x - mean and of its square.
__device__ __forceinline__ Stats moments(float mean, const float (&v)[2], float share, float eps) {
  Stats r = {mean, v[0] * share, 0.0f};
  r.rstd = rsqrtf(fmaxf(fmaf(v[1], share, -r.rest * r.rest), 0.0f) + eps);
  return r;
}

// A row's elements in the registers of `threads` threads, E each, 16 bytes of
// neighbours at a time: whole accesses (kWide: rows on 16 bytes, a whole number
// of accesses long) or, for the same bits, one by one (a warp's neighbours are
// then in L1).
template <class T, int E, bool kWide>
struct Held {
  static constexpr int V = 16 / sizeof(T);
  static constexpr int kPacks = E / V;
  static_assert(E % V == 0, "whole accesses");
  uint4 q[kWide ? kPacks : 1];
  T v[kWide ? 1 : E];

  static __device__ __forceinline__ int column(int e, int t, int threads) {
    return (e / V * threads + t) * V + e % V;
  }
  __device__ __forceinline__ void load(const T* p, int t, int threads, int dim) {
    if constexpr (kWide) {
#pragma unroll
      for (int k = 0; k < kPacks; ++k) {
        const int c = (k * threads + t) * V;
        q[k] = c < dim ? __ldcs(reinterpret_cast<const uint4*>(p + c)) : make_uint4(0, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = column(e, t, threads);
        v[e] = c < dim ? p[c] : from_f32<T>(0.0f);
      }
    }
  }
  __device__ __forceinline__ F2 pair(int i) const { return pack2(get(2 * i), get(2 * i + 1)); }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (kWide) {
      const uint4& w4 = q[e / V];
      const int i = e % V;
      if constexpr (sizeof(T) == 4) {
        return __uint_as_float(i == 0 ? w4.x : i == 1 ? w4.y : i == 2 ? w4.z : w4.w);
      } else {
        const uint32_t w = i / 2 == 0 ? w4.x : i / 2 == 1 ? w4.y : i / 2 == 2 ? w4.z : w4.w;
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
          return __uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16);
        else
          return __half2float(__ushort_as_half((unsigned short)(w >> (i % 2 * 16))));
      }
    } else {
      return to_f32(v[e]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const F2 (&pairs)[E / 2], int t, int threads,
                                               int dim) {
    float f[E];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) unpack2(pairs[i], f[2 * i], f[2 * i + 1]);
    if constexpr (kWide) {
#pragma unroll
      for (int k = 0; k < kPacks; ++k) {
        const int c = (k * threads + t) * V;
        if (c < dim) {
          float g[V];
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] = f[k * V + i];
          store_f32<T, V>(p + c, true, V, g);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = column(e, t, threads);
        if (c < dim) p[c] = from_f32<T>(f[e]);
      }
    }
  }
};

// Weights of a thread's columns (`none` without them, and behind the row).
template <int E, int V, bool kWide>
__device__ __forceinline__ void load_vector(const float* w, float none, int t, int threads, int dim,
                                            F2 (&pairs)[E / 2]) {
  float f[E];
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = none;
  if (w != nullptr) {
  if constexpr (kWide) {
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
      const int c = (k * threads + t) * V;
      if (c < dim) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(w + c + i));
          f[k * V + i] = q.x, f[k * V + i + 1] = q.y;
          f[k * V + i + 2] = q.z, f[k * V + i + 3] = q.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e / V * threads + t) * V + e % V;
      if (c < dim) f[e] = __ldg(w + c);
    }
  }
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) pairs[i] = pack2(f[2 * i], f[2 * i + 1]);
}

// The threads of a row: whole warps of a block.
struct Team {
  int threads, t;  // and this one's number
  int warps, first;  // its warps, and the one that this lane adds up
  bool full;         // whether all elements of this warp lie inside the row
  __device__ Team(int threads_, int dim, int V, int packs) : threads(threads_) {
    t = threadIdx.x % threads;
    warps = threads / 32;
    first = threadIdx.x / threads * warps + threadIdx.x % 32 % warps;
    full = __all_sync(~0u, ((packs - 1) * threads + t) * V + V <= dim);
  }
};

// Sums of N numbers over the threads of a row, in one order: by lanes, then by
// warps, whose sums every warp adds up in the same tree. buf: N numbers a warp,
// not in use.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], const Team& team, float (*buf)[32]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if (team.warps == 1) return;
  if (threadIdx.x % 32 == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) buf[k][threadIdx.x / 32] = v[k];
  }
  __syncthreads();
  // (lanes read the row's warps over and over: a tree of warps in every lane)
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = buf[k][team.first];
#pragma unroll
  for (int s = 16; s > 0; s /= 2) {
    if (s >= team.warps) continue;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __fadd_rn(v[k], __shfl_xor_sync(~0u, v[k], s));
  }
}
__device__ __forceinline__ float both(F2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return __fadd_rn(lo, hi);
}

// Zeros what is behind the row.
template <class H, int N>
__device__ __forceinline__ void clip(F2 (&d)[N], const Team& team, int dim) {
  if (team.full) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float lo, hi;
    unpack2(d[i], lo, hi);
    d[i] = pack2(H::column(2 * i, team.t, team.threads) < dim ? lo : 0.0f,
                 H::column(2 * i + 1, team.t, team.threads) < dim ? hi : 0.0f);
  }
}

// The statistics of a row whose elements are x; leaves x - mean in d.
template <class T, int E, bool kWide>
__device__ __forceinline__ Stats row_stats(const Held<T, E, kWide>& x, const Team& team, int dim,
                                           float share, float eps, float (*buf)[32],
                                           F2 (&d)[E / 2]) {
  F2 s = 0, s2 = 0;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    d[i] = x.pair(i);
    s = add2(s, d[i]);
  }
  float m[1] = {both(s)};
  row_sum(m, team, buf);
  const float mean = m[0] * share;
  const F2 minus = pack2(-mean, -mean);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) d[i] = add2(d[i], minus);
  clip<Held<T, E, kWide>>(d, team, dim);
  s = 0;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    s = add2(s, d[i]);
    s2 = fma2(d[i], d[i], s2);
  }
  float v[2] = {both(s), both(s2)};
  row_sum(v, team, buf + 1);
  return moments(mean, v, share, eps);
}

// A row in the registers of `threads` threads, several rows a block, which walks
// rows `blocks` apart, the next one's elements in flight. y NULL: the statistics
// alone.
template <class T, int kThreads, int E, bool kWide>
__global__ void __launch_bounds__(kThreads)
layer_norm_kernel(NormIn<T> in, int threads, T* __restrict__ y, Rows2 ys,
                  float* __restrict__ stats) {
  using H = Held<T, E, kWide>;
  __shared__ float buf[2][3][32];
  const int dim = (int)in.dim;
  const Team team(threads, dim, H::V, E / H::V);
  const int t = team.t, groups = kThreads / threads;
  const float share = 1.0f / (float)dim;
  const int64_t step = (int64_t)gridDim.x * groups;
  // 1024 threads have 64 registers each: no room for the next row, nor to keep
  // the weights
  constexpr bool kLean = kThreads == 1024;
  F2 w[E / 2], b[E / 2];
  if constexpr (!kLean) {
    load_vector<E, H::V, kWide>(in.w, 1.0f, t, threads, dim, w);
    load_vector<E, H::V, kWide>(in.b, 0.0f, t, threads, dim, b);
  }
  H next;
  const auto fetch = [&](int64_t r) {
    const bool real = r < in.rows;
    next.load(in.x + row_offset(real ? r : 0, in.len, in.xs), t, threads, real ? dim : 0);
  };
  int64_t r = (int64_t)blockIdx.x * groups + threadIdx.x / threads;
  if (!kLean) fetch(r);
  // (as many turns for all rows of a block: they wait for one another)
  for (int64_t r0 = (int64_t)blockIdx.x * groups, turn = 0; r0 < in.rows; r0 += step, ++turn) {
    if (kLean) fetch(r);
    const H x = next;
    const int64_t now = r;
    r += step;
    if (!kLean && r0 + step < in.rows) fetch(r);
    F2 d[E / 2];
    const Stats st = row_stats(x, team, dim, share, in.eps, buf[turn & 1], d);
    if (now >= in.rows) continue;
    if (stats != nullptr && t == 0) {
      stats[3 * now] = st.mean;
      stats[3 * now + 1] = st.rest;
      stats[3 * now + 2] = st.rstd;
    }
    if (y == nullptr) continue;
    if constexpr (kLean) {
      load_vector<E, H::V, kWide>(in.w, 1.0f, t, threads, dim, w);
      load_vector<E, H::V, kWide>(in.b, 0.0f, t, threads, dim, b);
    }
    const F2 rstd = pack2(st.rstd, st.rstd);
    const F2 shift = pack2(-st.rest * st.rstd, -st.rest * st.rstd);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) d[i] = fma2(fma2(d[i], rstd, shift), w[i], b[i]);
    H::store(y + row_offset(now, in.len, ys), d, t, threads, dim);
  }
}

// Rows that registers do not hold: a block a row, read again from L2.
constexpr int kLongThreads = 512;
template <class T>
__device__ Stats long_stats(const T* x, int64_t dim, float eps, float (*buf)[32]) {
  const float share = 1.0f / (float)dim;
  float s[1] = {0.0f};
  for (int64_t c = threadIdx.x; c < dim; c += kLongThreads) s[0] += to_f32(x[c]);
  const Team team(kLongThreads, 0, 1, 1);
  row_sum(s, team, buf);
  const float mean = s[0] * share;
  float v[2] = {0.0f, 0.0f};
  for (int64_t c = threadIdx.x; c < dim; c += kLongThreads) {
    const float d = to_f32(x[c]) - mean;
    v[0] += d;
    v[1] = fmaf(d, d, v[1]);
  }
  row_sum(v, team, buf + 1);
  return moments(mean, v, share, eps);
}

template <class T>
__global__ void __launch_bounds__(kLongThreads)
layer_norm_long_kernel(NormIn<T> in, T* __restrict__ y, Rows2 ys, float* __restrict__ stats) {
  __shared__ float buf[3][32];
  const int64_t r = blockIdx.x;
  const T* x = in.x + row_offset(r, in.len, in.xs);
  const Stats st = long_stats(x, in.dim, in.eps, buf);
  T* yr = y + row_offset(r, in.len, ys);
  for (int64_t c = threadIdx.x; y != nullptr && c < in.dim; c += kLongThreads) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float w = in.w != nullptr ? in.w[c] : 1.0f, b = in.b != nullptr ? in.b[c] : 0.0f;
    yr[c] = from_f32<T>(fmaf(n, w, b));
  }
  if (stats != nullptr && threadIdx.x == 0) {
    stats[3 * r] = st.mean;
    stats[3 * r + 1] = st.rest;
    stats[3 * r + 2] = st.rstd;
  }
}

// dx, and a block's part of the sums over rows, in registers: a block walks
// rows `blocks` apart, the next one's elements in flight. part: [block][2][dim].
template <class T, int kThreads, int E, bool kWide>
__global__ void __launch_bounds__(kThreads)
layer_norm_backward_kernel(NormIn<T> in, int threads, const T* __restrict__ dy, Rows2 ds,
                           const float* __restrict__ stats, T* __restrict__ dx, Rows2 os,
                           float* __restrict__ part) {
  using H = Held<T, E, kWide>;
  __shared__ float buf[2][5][32];
  extern __shared__ float sums[];  // [2][dim], for several rows a block
  const int dim = (int)in.dim;
  const Team team(threads, dim, H::V, E / H::V);
  const int t = team.t, groups = kThreads / threads, group = threadIdx.x / threads;
  const int64_t step = (int64_t)gridDim.x * groups;
  const float share = 1.0f / (float)dim;
  F2 w[E / 2], dw[E / 2], db[E / 2];
  load_vector<E, H::V, kWide>(in.w, 1.0f, t, threads, dim, w);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dw[i] = db[i] = 0;
  H x, g;
  Stats next = {0.0f, 0.0f, 0.0f};
  const auto fetch = [&](int64_t r) {
    const bool real = r < in.rows;
    x.load(in.x + row_offset(real ? r : 0, in.len, in.xs), t, threads, real ? dim : 0);
    g.load(dy + row_offset(real ? r : 0, in.len, ds), t, threads, real ? dim : 0);
    if (stats != nullptr && real)
      next = {__ldg(stats + 3 * r), __ldg(stats + 3 * r + 1), __ldg(stats + 3 * r + 2)};
  };
  int64_t r = (int64_t)blockIdx.x * groups + group;
  fetch(r);
  // (as many turns for all rows of a block: they wait for one another)
  for (int64_t r0 = (int64_t)blockIdx.x * groups, turn = 0; r0 < in.rows; r0 += step, ++turn) {
    float(*const b)[32] = buf[turn & 1];
    F2 n[E / 2], q[E / 2];
    Stats st = next;
    if (stats == nullptr) {
      st = row_stats(x, team, dim, share, in.eps, b, n);
    } else {
      const F2 minus = pack2(-st.mean, -st.mean);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) n[i] = add2(x.pair(i), minus);
    }
    const F2 rstd = pack2(st.rstd, st.rstd);
    const F2 shift = pack2(-st.rest * st.rstd, -st.rest * st.rstd);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) n[i] = fma2(n[i], rstd, shift);
    clip<H>(n, team, dim);
    F2 s1 = 0, s2 = 0;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const F2 u = g.pair(i);
      dw[i] = fma2(u, n[i], dw[i]);
      db[i] = add2(db[i], u);
      q[i] = mul2(u, w[i]);
      s1 = fma2(u, w[i], s1);  // (a sum of q, which add2 is not for)
      s2 = fma2(q[i], n[i], s2);
    }
    const int64_t now = r;
    r += step;
    fetch(r);
    float v[2] = {both(s1), both(s2)};
    row_sum(v, team, b + 3);
    if (now < in.rows) {
      const float a1 = v[0] * share * -st.rstd, a2 = v[1] * share * -st.rstd;
      const F2 p1 = pack2(a1, a1), p2 = pack2(a2, a2);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) q[i] = fma2(n[i], p2, fma2(q[i], rstd, p1));
      H::store(dx + row_offset(now, in.len, os), q, t, threads, dim);
    }
  }
  float dw1[E], db1[E];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    unpack2(dw[i], dw1[2 * i], dw1[2 * i + 1]);
    unpack2(db[i], db1[2 * i], db1[2 * i + 1]);
  }
  float* const out = part + (int64_t)blockIdx.x * 2 * dim;
  if (groups == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = H::column(e, t, threads);
      if (c < dim) out[c] = dw1[e], out[dim + c] = db1[e];
    }
    return;
  }
  for (int k = 0; k < groups; ++k) {  // group by group, in order
    if (group == k) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = H::column(e, t, threads);
        if (c < dim) {
          sums[c] = k == 0 ? dw1[e] : sums[c] + dw1[e];
          sums[dim + c] = k == 0 ? db1[e] : sums[dim + c] + db1[e];
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * dim; c += kThreads) out[c] = sums[c];
}

// Long rows: dx alone.
template <class T>
__global__ void __launch_bounds__(kLongThreads)
layer_norm_backward_long_kernel(NormIn<T> in, const T* __restrict__ dy, Rows2 ds,
                                const float* __restrict__ stats, T* __restrict__ dx, Rows2 os) {
  __shared__ float buf[2][32];
  const int64_t r = blockIdx.x;
  const T* x = in.x + row_offset(r, in.len, in.xs);
  const T* d = dy + row_offset(r, in.len, ds);
  const Stats st = {stats[3 * r], stats[3 * r + 1], stats[3 * r + 2]};
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = threadIdx.x; c < in.dim; c += kLongThreads) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float g = to_f32(d[c]) * (in.w != nullptr ? in.w[c] : 1.0f);
    s1 += g;
    s2 = fmaf(g, n, s2);
  }
  float v[2] = {s1, s2};
  row_sum(v, Team(kLongThreads, 0, 1, 1), buf);
  const float a1 = v[0] / (float)in.dim, a2 = v[1] / (float)in.dim;
  T* o = dx + row_offset(r, in.len, os);
  for (int64_t c = threadIdx.x; c < in.dim; c += kLongThreads) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float g = to_f32(d[c]) * (in.w != nullptr ? in.w[c] : 1.0f);
    o[c] = from_f32<T>(st.rstd * fmaf(-n, a2, g - a1));
  }
}

constexpr int kSumRows = 256;  // rows of a partial sum of long rows

template <class T>
__global__ void __launch_bounds__(256)
layer_norm_part_kernel(NormIn<T> in, const T* __restrict__ dy, Rows2 ds,
                       const float* __restrict__ stats, float* __restrict__ part) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= in.dim) return;
  for (int64_t p = blockIdx.y; p * kSumRows < in.rows; p += gridDim.y) {
    float dw = 0.0f, db = 0.0f;
    const int64_t end = min(in.rows, (p + 1) * kSumRows);
#pragma unroll 4
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

// The sums of the parts: a block 32 columns, a warp every 32nd part, then the
// warps in order.
__global__ void __launch_bounds__(1024)
layer_norm_sum_kernel(const float* __restrict__ part, int64_t parts, int64_t dim,
                      float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float buf[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;  // of 2 dim
  float v = 0.0f;
  if (c < 2 * dim) {
#pragma unroll 8
    for (int64_t p = warp; p < parts; p += 32) v += __ldg(part + p * 2 * dim + c);
  }
  buf[warp][lane] = v;
  __syncthreads();
  if (warp != 0) return;
  v = buf[0][lane];
#pragma unroll
  for (int w = 1; w < 32; ++w) v += buf[w][lane];
  if (c < dim) {
    if (dw != nullptr) dw[c] = v;
  } else if (c < 2 * dim) {
    if (db != nullptr) db[c - dim] = v;
  }
}

// (A batch whose rows are evenly spaced is one sequence: its strides and all
// others' are then the time strides alone.)
bool even(int64_t batch, int64_t len, Rows2 s) { return batch <= 1 || s.bs == len * s.ts; }

template <class T>
NormIn<T> norm_in(const cr_layer_norm_args* a, bool one_batch) {
  return {a->batch * a->len, one_batch ? 0 : a->len, a->dim, a->eps, static_cast<const T*>(a->x),
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

// How rows lie in threads: by their length alone, so that a row's bits are the
// same among any others and in both directions.
struct NormShape {
  int block;    // threads of a block
  int threads;  // of a row, 0: more than registers hold
  int E;        // elements a thread
};

NormShape norm_shape(int64_t dim) {
  NormShape sh = {256, 0, 8};
  if (dim > 16384) return sh;
  if (dim > 2048) sh.block = 512;
  if (dim > 4096) sh.E = 16;
  if (dim > 8192) sh.block = 1024;
  sh.threads = 32;
  while ((int64_t)sh.threads * sh.E < dim) sh.threads *= 2;
  return sh;
}

// Blocks of the backward call, which leave a part of the sums over rows each; 0:
// rows whose gradient goes another way.
#ifndef CR_NORM_BLOCKS
#define CR_NORM_BLOCKS 456
#endif
int64_t norm_blocks(int64_t rows, int64_t dim) {
  if (dim > 8192) return 0;
  const NormShape sh = norm_shape(dim);
  const int64_t most = sh.block == 256 ? CR_NORM_BLOCKS : sh.E == 8 ? 304 : 152;
  return std::min<int64_t>(ceil_div(rows, sh.block / sh.threads), most);
}

bool norm_wide(const cr_layer_norm_args* a) {
  const size_t es = model_esize(a->dt);
  return a->dim % (int64_t)(16 / es) == 0 &&
         rows_aligned(a->x, a->x_batch_stride, a->x_time_stride, es, 16) &&
         ptr_aligned(a->weight, 16) && ptr_aligned(a->bias, 16);
}

// Runs EXPR with a block's threads B, a thread's elements E and the access W.
#define CR_NORM_CASE(B_, E_, WIDE, ...)                                       \
  {                                                                           \
    constexpr int B = B_, E = E_;                                             \
    if (WIDE) { constexpr bool W = true; __VA_ARGS__; }                       \
    else { constexpr bool W = false; __VA_ARGS__; }                           \
  }
#define CR_NORM_SHAPE(SH, WIDE, ...)                                          \
  if (SH.block == 1024) CR_NORM_CASE(1024, 16, WIDE, __VA_ARGS__)             \
  else CR_NORM_BACKWARD_SHAPE(SH, WIDE, __VA_ARGS__)
#define CR_NORM_BACKWARD_SHAPE(SH, WIDE, ...)                                 \
  if (SH.E == 16) CR_NORM_CASE(512, 16, WIDE, __VA_ARGS__)                    \
  else if (SH.block == 512) CR_NORM_CASE(512, 8, WIDE, __VA_ARGS__)           \
  else CR_NORM_CASE(256, 8, WIDE, __VA_ARGS__)

#ifndef CR_NORM_RES
#define CR_NORM_RES(B) (1024 / (B))
#endif
void launch_norm(const cr_layer_norm_args* a, void* y, Rows2 ys, float* stats, bool wide,
                 cudaStream_t s) {
  const NormShape sh = norm_shape(a->dim);
  const int64_t rows = a->batch * a->len;
  const Rows2 xs = {a->x_batch_stride, a->x_time_stride};
  const bool one = even(a->batch, a->len, xs) && even(a->batch, a->len, ys);
  CR_MODEL_TYPE(a->dt, {
    T* out = static_cast<T*>(y);
    if (sh.threads == 0) {
      CR_LAUNCH(kKLayerNorm, s,
                layer_norm_long_kernel<T><<<(unsigned)rows, kLongThreads, 0, s>>>(norm_in<T>(a, one), out,
                                                                                  ys, stats));
    } else {
      CR_NORM_SHAPE(sh, wide, {
        CR_LAUNCH(kKLayerNorm, s,
                  layer_norm_kernel<T, B, E, W>
                  <<<(unsigned)std::min<int64_t>(ceil_div(rows, B / sh.threads), 152 * CR_NORM_RES(B)), B,
                     0, s>>>(norm_in<T>(a, one), sh.threads, out, ys, stats));
      });
    }
  });
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
  const Rows2 ys = {y_batch_stride, y_time_stride};
  const bool wide = norm_wide(a) && rows_aligned(y, y_batch_stride, y_time_stride, es, 16);
  launch_norm(a, y, ys, stats, wide, s);
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

size_t cr_layer_norm_backward_workspace_bytes(int64_t batch, int64_t len, int64_t dim) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || (len > 0 && batch > kMaxBlocks / len)) return 0;
  const int64_t rows = batch * len;
  const int64_t blocks = norm_blocks(rows, dim);
  const size_t parts = (size_t)(blocks != 0 ? blocks : ceil_div(rows, kSumRows));
  return (blocks != 0 ? 0 : round256((size_t)rows * 12)) + round256(parts * dim * 8) +
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
  const Rows2 ds = {g->dy_batch_stride, g->dy_time_stride};
  const Rows2 os = {g->dx_batch_stride, g->dx_time_stride};
  const NormShape sh = norm_shape(a->dim);
  const int64_t blocks = norm_blocks(rows, a->dim);
  const bool wide = norm_wide(a) &&
                    rows_aligned(g->dy, g->dy_batch_stride, g->dy_time_stride, es, 16) &&
                    rows_aligned(g->dx, g->dx_batch_stride, g->dx_time_stride, es, 16);
  const int64_t sum_blocks = ceil_div(2 * a->dim, 32), cols = ceil_div(a->dim, 256);
  if (sum_blocks > kMaxBlocks) return CR_ERR_UNSUPPORTED;
  char* at = past_status(ws);
  float* kept = reinterpret_cast<float*>(at);
  if (blocks == 0) at += round256((size_t)rows * 12);
  float* part = reinterpret_cast<float*>(at);
  const int64_t parts = blocks != 0 ? blocks : ceil_div(rows, kSumRows);
  const float* stats = g->stats;
  if (rows > 0 && blocks == 0 && stats == nullptr) {
    launch_norm(a, nullptr, {a->x_batch_stride, a->x_time_stride}, kept, norm_wide(a), s);
    stats = kept;
  }
  const Rows2 xs = {a->x_batch_stride, a->x_time_stride};
  const bool one = even(a->batch, a->len, xs) && even(a->batch, a->len, ds) &&
                   even(a->batch, a->len, os);
  CR_MODEL_TYPE(a->dt, {
    const T* dy = static_cast<const T*>(g->dy);
    T* dx = static_cast<T*>(g->dx);
    if (rows > 0 && blocks == 0) {
      CR_LAUNCH(kKLayerNormBackward, s,
                layer_norm_backward_long_kernel<T><<<(unsigned)rows, kLongThreads, 0, s>>>(
                    norm_in<T>(a, one), dy, ds, stats, dx, os));
      CR_LAUNCH(kKLayerNormSum, s,
                layer_norm_part_kernel<T>
                <<<dim3((unsigned)cols, (unsigned)std::min<int64_t>(parts, 65535)), 256, 0, s>>>(
                    norm_in<T>(a, one), dy, ds, stats, part));
    } else if (rows > 0) {
      CR_NORM_BACKWARD_SHAPE(sh, wide, {
        const size_t smem = sh.threads < B ? (size_t)a->dim * 8 : 0;
        CR_LAUNCH(kKLayerNormBackward, s,
                  layer_norm_backward_kernel<T, B, E, W><<<(unsigned)blocks, B, smem, s>>>(
                      norm_in<T>(a, one), sh.threads, dy, ds, stats, dx, os, part));
      });
    }
    if (g->dweight != nullptr || g->dbias != nullptr)
      CR_LAUNCH(kKLayerNormSum, s,
                layer_norm_sum_kernel<<<(unsigned)sum_blocks, 1024, 0, s>>>(part, parts, a->dim,
                                                                            g->dweight, g->dbias));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
