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
  const T* end;  // of x
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

// The threads of a row: whole warps of a block.
struct Team {
  int threads, t;    // and this one's number
  int warps, first;  // its warps, and the one that this lane adds up
  __device__ explicit Team(int threads_) : threads(threads_) {
    t = threadIdx.x % threads;
    warps = threads / 32;
    first = threadIdx.x / threads * warps + threadIdx.x % 32 % warps;
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
  for (int s = team.warps / 2; s > 0; s /= 2) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __fadd_rn(v[k], __shfl_xor_sync(~0u, v[k], s));
  }
}
__device__ __forceinline__ float both(F2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return __fadd_rn(lo, hi);
}

// How rows move: where they lie on 16 bytes and are a whole number of those
// long, by these (kWhole). Otherwise by the places of 16 bytes that they lie in
// (kPlaces, Ragged), or, short ones, element by element (kElements): places cost a
// row more, and its elements less. All give the same bits.
enum Move { kElements, kPlaces, kWhole };

// 16 bytes of neighbours.
template <class T>
struct Quad {
  static constexpr int V = 16 / sizeof(T);
  uint4 q;
  // One by one (a warp's neighbours are then in L1); have: elements inside the row.
  __device__ __forceinline__ void load(const T* p, int have) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i >= have) continue;
      if constexpr (sizeof(T) == 4) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
      else
        w[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << i % 2 * 16;
    }
    q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store(T* p, const F2 (&v)[V / 2], int have) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
    store_f32<T, V>(p, false, have, f);
  }
  __device__ __forceinline__ F2 pair(int i) const {
    if constexpr (sizeof(T) == 4) {
      return i == 0 ? pack2(__uint_as_float(q.x), __uint_as_float(q.y))
                    : pack2(__uint_as_float(q.z), __uint_as_float(q.w));
    } else {
      const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return pack2(f.x, f.y);
      }
    }
  }
  __device__ __forceinline__ static uint4 packed(const F2 (&v)[V / 2]) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      float lo, hi;
      unpack2(v[i], lo, hi);
      r.v[2 * i] = from_f32<T>(lo);
      r.v[2 * i + 1] = from_f32<T>(hi);
    }
    return __builtin_bit_cast(uint4, r);
  }
};

// Rows that start anywhere or have no whole number of 16 bytes move by the 16-byte
// places that they lie in, of which the first and the last may be shared with what
// is beside the row. In shared memory a row lies in the same places, `shift`
// elements off, and is put right by whoever reads it; a result is put in its
// places as it is stored. (Loaded and stored element by element, eight a lane,
// 16,384 rows of 2049 in bf16 took 110 us, their gradient 166; by words of 4 bytes
// 98 and 193.)
template <class T>
struct Ragged {
  static constexpr int V = 16 / sizeof(T), kHalves = 4 / sizeof(T);
  using Elements = Pack<T, V>;
  static __device__ __forceinline__ int shift(const T* p) {
    return (int)((uintptr_t)p % 16) / (int)sizeof(T);
  }
  // The row of dim elements at p into `to` (one place more than its own 16 bytes
  // may take), by thread t of several. lo and hi: where the tensor begins and
  // ends, beyond which nothing is read.
  static __device__ __forceinline__ void fetch(uint4* to, const T* p, int dim, const T* lo,
                                               const T* hi, int t, int threads) {
    const int s = shift(p), n = (dim + s + V - 1) / V;
    const T* const a = p - s;
    const bool inside = a >= lo && a + n * V <= hi;
#pragma unroll 2
    for (int q = t; q < n; q += threads) {
      const int e = q * V;
      if (inside || (a + e >= lo && a + e + V <= hi)) {
        copy16(to + q, a + e);
      } else {
        Elements v;
#pragma unroll
        for (int i = 0; i < V; ++i)
          v.v[i] = e + i >= s && e + i - s < dim ? p[e + i - s] : from_f32<T>(0.0f);
        to[q] = __builtin_bit_cast(uint4, v);
      }
    }
  }
  // The 16 bytes that begin s elements into a.
  static __device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int s) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int words = s / kHalves;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = words & 2 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
    if constexpr (kHalves == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], s % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Elements q V to q V + V of a row in shared memory; zeros from `have` of them on.
  static __device__ __forceinline__ uint4 quad(const uint4* row, int q, int s, int have) {
    if (have <= 0) return make_uint4(0, 0, 0, 0);
    const uint4 r = s == 0 ? row[q] : shifted(row[q], row[q + 1], s);
    if (have >= V) return r;
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = have - i * kHalves;
      w[i] = left <= 0 ? 0u : left < kHalves ? w[i] & 0xFFFFu : w[i];
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // A row that lies unshifted in shared memory (and a place behind it) to p, by
  // thread t of at least 8: the elements before and after its whole places one by
  // one.
  static __device__ __forceinline__ void store(T* p, const uint4* row, int dim, int t,
                                               int threads) {
    const int head = min((V - shift(p)) % V, dim), full = (dim - head) / V;
    const int done = head + full * V;
    const T* const e = reinterpret_cast<const T*>(row);
    if (t < head) p[t] = e[t];
    if (t < dim - done) p[done + t] = e[done + t];
    uint4* const to = reinterpret_cast<uint4*>(p + head);
#pragma unroll 2
    for (int q = t; q < full; q += threads)
      to[q] = head == 0 ? row[q] : shifted(row[q], row[q + 1], head);
  }
};
// The same of weights, V floats on 16 bytes; `none` without them.
template <int V, bool kWide>
__device__ __forceinline__ void load_vector(const float* w, int c, int have, float none,
                                            F2 (&v)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) v[i] = pack2(none, none);
  if (w == nullptr) return;
  if constexpr (kWide) {
    if (have > 0) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(w + c + i));
        v[i / 2] = pack2(q.x, q.y);
        v[i / 2 + 1] = pack2(q.z, q.w);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      v[i] = pack2(2 * i < have ? __ldg(w + c + 2 * i) : none,
                   2 * i + 1 < have ? __ldg(w + c + 2 * i + 1) : none);
  }
}
// Zeros what is behind the row.
template <int N>
__device__ __forceinline__ void clip(F2 (&d)[N], int have) {
  if (have >= 2 * N) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float lo, hi;
    unpack2(d[i], lo, hi);
    d[i] = pack2(2 * i < have ? lo : 0.0f, 2 * i + 1 < have ? hi : 0.0f);
  }
}

// A row a warp, or several warps a row: a lane has kQuads times 16 bytes, so that
// what a row costs besides its elements, sums over lanes above all, is shared by
// many of them, and few rows wait at a barrier. Rows come by way of shared
// memory, each thread's own part of it, two rows ahead, and stay there as they
// stand in memory; the weights stand beside them. y NULL: the statistics alone.
constexpr int kNormThreads = 256;
// Bytes of the rows: [turn][row][quad], a place more a row with kPlaces.
template <int kQuads, Move kMove>
__host__ __device__ constexpr size_t norm_rows_bytes(int groups) {
  return sizeof(uint4) * 2 * (kQuads * kNormThreads + (kMove == kPlaces ? groups : 0));
}
template <class T, int kQuads, Move kMove>
__global__ void __launch_bounds__(kNormThreads)
layer_norm_kernel(NormIn<T> in, int threads, T* __restrict__ y, Rows2 ys,
                  float* __restrict__ stats) {
  constexpr bool kWide = kMove == kWhole;
  using Q = Quad<T>;
  using R = Ragged<T>;
  constexpr int V = Q::V, N = V / 2;
  __shared__ float buf[2][3][32];
  extern __shared__ __align__(16) char shared[];
  const int dim = (int)in.dim, columns = kQuads * threads * V;
  const Team team(threads);
  const int groups = kNormThreads / threads;
  const int64_t step = (int64_t)gridDim.x * groups;
  const int group = threadIdx.x / threads, pitch = kQuads * threads + (kMove == kPlaces);
  const auto row = [&](int turn) {
    return reinterpret_cast<uint4*>(shared) + (turn * groups + group) * pitch;
  };
  // Weights and biases, four columns of a lane at a time, so that a warp's
  // accesses are consecutive: [2][quad][V / 4][thread].
  float4* const weights =
      reinterpret_cast<float4*>(shared + norm_rows_bytes<kQuads, kMove>(groups));
  const auto column = [&](int k) { return (k * threads + team.t) * V; };
  const auto fetch = [&](int64_t r, int turn) {
    if (r < in.rows) {
      const T* p = in.x + row_offset(r, in.len, in.xs);
      if constexpr (kWide) {
#pragma unroll
        for (int k = 0; k < kQuads; ++k)
          if (column(k) < dim) copy16(row(turn) + k * threads + team.t, p + column(k));
      } else if constexpr (kMove == kElements) {
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
          Q q;
          q.load(p + column(k), dim - column(k));
          row(turn)[k * threads + team.t] = q.q;
        }
      } else {
        R::fetch(row(turn), p, dim, in.x, in.end, team.t, threads);
      }
    }
    copy_commit();
  };
  const auto wait_for_team = [&] {
    if (team.warps == 1) __syncwarp();
    else __syncthreads();
  };
  int64_t r = (int64_t)blockIdx.x * groups + group;
  if (kMove != kPlaces && column(kQuads - 1) >= dim) {  // what no row fills
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
      if (column(k) >= dim)
        row(0)[k * threads + team.t] = row(1)[k * threads + team.t] = make_uint4(0, 0, 0, 0);
  }
  fetch(r, 0);
  fetch(r + step, 1);
  if (y != nullptr) {
    // (threads is a power of two; V / 4 accesses a quad)
    constexpr int kParts = V / 4;
    const int bits = 31 - __clz(threads);
#pragma unroll 4
    for (int i = threadIdx.x; i < columns / 4; i += kNormThreads) {
      const int t = i & (threads - 1), four = i >> bits;
      const int c = (four / kParts * threads + t) * V + four % kParts * 4;
      F2 w[2], b[2];
      load_vector<4, kWide>(in.w, c, dim - c, 1.0f, w);
      load_vector<4, kWide>(in.b, c, dim - c, 0.0f, b);
      float4 f;
      unpack2(w[0], f.x, f.y);
      unpack2(w[1], f.z, f.w);
      weights[i] = f;
      unpack2(b[0], f.x, f.y);
      unpack2(b[1], f.z, f.w);
      weights[columns / 4 + i] = f;
    }
  }
  __syncthreads();
  const float share = 1.0f / (float)dim;
  // (as many turns for all rows of a block: they may wait for one another)
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < in.rows;
       r0 += step, r += step, turn ^= 1) {
    copy_wait<1>();
    Q q[kQuads];
    if constexpr (kMove != kPlaces) {
#pragma unroll
      for (int k = 0; k < kQuads; ++k) q[k].q = row(turn)[k * threads + team.t];
      fetch(r + 2 * step, turn);
    } else {
      wait_for_team();
      const int shift = R::shift(in.x + row_offset(r < in.rows ? r : 0, in.len, in.xs));
#pragma unroll
      for (int k = 0; k < kQuads; ++k)
        q[k].q = R::quad(row(turn), k * threads + team.t, shift,
                         r < in.rows ? dim - column(k) : 0);
      wait_for_team();  // (y takes the row's place)
    }
    F2 s[2] = {0, 0}, s2[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i % 2] = add2(s[i % 2], q[k].pair(i));
    float m[1] = {both(add2(s[0], s[1]))};
    row_sum(m, team, buf[turn]);
    const float mean = m[0] * share;
    const F2 minus = pack2(-mean, -mean);
    s[0] = s[1] = 0;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      F2 d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = add2(q[k].pair(i), minus);
      clip(d, dim - column(k));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[i % 2] = add2(s[i % 2], d[i]);
        s2[i % 2] = fma2(d[i], d[i], s2[i % 2]);
      }
    }
    float v[2] = {both(add2(s[0], s[1])), both(s2[0]) + both(s2[1])};
    row_sum(v, team, buf[turn] + 1);
    const Stats st = moments(mean, v, share, in.eps);
    if (r < in.rows && stats != nullptr && team.t == 0) {
      stats[3 * r] = st.mean;
      stats[3 * r + 1] = st.rest;
      stats[3 * r + 2] = st.rstd;
    }
    if (r < in.rows && y != nullptr) {
      const F2 rstd = pack2(st.rstd, st.rstd);
      const F2 shift = pack2(-st.rest * st.rstd, -st.rest * st.rstd);
      T* out = y + row_offset(r, in.len, ys);
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int c = column(k), have = dim - c;
        F2 o[N];
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const int at = (k * (V / 4) + i / 2) * threads + team.t;
          const float4 w = weights[at], b = weights[columns / 4 + at];
          o[i] = fma2(fma2(add2(q[k].pair(i), minus), rstd, shift), pack2(w.x, w.y),
                      pack2(b.x, b.y));
          o[i + 1] = fma2(fma2(add2(q[k].pair(i + 1), minus), rstd, shift), pack2(w.z, w.w),
                          pack2(b.z, b.w));
        }
        if constexpr (kWide) {
          if (have > 0) *reinterpret_cast<uint4*>(out + c) = Q::packed(o);
        } else if constexpr (kMove == kElements) {
          if (have > 0) Q::store(out + c, o, have);
        } else {
          row(turn)[k * threads + team.t] = Q::packed(o);
        }
      }
    }
    if constexpr (kMove == kPlaces) {
      if (y != nullptr) {
        wait_for_team();
        if (r < in.rows)
          R::store(y + row_offset(r, in.len, ys), row(turn), dim, team.t, threads);
        wait_for_team();
      }
      fetch(r + 2 * step, turn);
    }
  }
  copy_wait<0>();
}

// Rows that registers do not hold: a block a row, read again from L2.
constexpr int kLongThreads = 512;
template <class T>
__device__ Stats long_stats(const T* x, int64_t dim, float eps, float (*buf)[32]) {
  const float share = 1.0f / (float)dim;
  float s[1] = {0.0f};
  for (int64_t c = threadIdx.x; c < dim; c += kLongThreads) s[0] += to_f32(x[c]);
  const Team team(kLongThreads);
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

// The sums of p and of q over a warp, each in half of the lanes.
__device__ __forceinline__ float warp_sum2(float p, float q) {
  const bool up = threadIdx.x % 32 & 16;
  float c = up ? q : p;
  c = __fadd_rn(c, __shfl_xor_sync(~0u, up ? p : q, 16));
#pragma unroll
  for (int s = 8; s > 0; s /= 2) c = __fadd_rn(c, __shfl_xor_sync(~0u, c, s));
  return c;
}

// dx, and a block's part of the sums over rows, in registers. A turn is a few
// rows, held in shared memory, where the next turn's rows are on their way. A
// warp first takes a row, or a part of one, for its two sums; then a thread takes
// its columns of the rows. So what a row costs besides its elements is shared by
// many, and the block waits twice a turn, not for each row. (With all of a block's
// threads on one row, four rows ahead, the gradient of 16,384 x 2048 in bf16 took
// 60 us, its sums included; this takes 52, 57 % of the copy rate. Three blocks an SM
// for two: 54; four turns held for two: 53 to 56.) part: [block][2][dim], or NULL.
template <int kThreads, int kRows>
struct Turn {
  static constexpr int kWarps = kThreads / 32 / kRows;  // of a row
  float sums[kRows][2][kWarps];
  float stats[2][kRows][3];  // turn
  int shift[2][kRows][2];    // of x and dy, with kPlaces
};
template <class T, int kThreads, int kQuads, int kRows, Move kMove>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1)
layer_norm_backward_kernel(NormIn<T> in, int threads, const T* __restrict__ dy, Rows2 ds,
                           const T* __restrict__ dy_end, const float* __restrict__ stats,
                           T* __restrict__ dx, Rows2 os, float* __restrict__ part) {
  constexpr bool kWide = kMove == kWhole;
  using Q = Quad<T>;
  using R = Ragged<T>;
  constexpr int V = Q::V, N = V / 2, W = Turn<kThreads, kRows>::kWarps;
  __shared__ Turn<kThreads, kRows> sh;
  // uint4 [turn][row][x or dy][quad], and dx [row][quad] with kPlaces, float4 [V /
  // 4][quad] of weights; at the end sums [2][dim]. (With kPlaces a place more a row.)
  extern __shared__ __align__(16) char shared[];
  const int dim = (int)in.dim, quads = (dim + V - 1) / V;
  uint4* const held = reinterpret_cast<uint4*>(shared);
  const int pitch = quads + (kMove == kPlaces);
  uint4* const results = held + 4 * kRows * pitch;
  float4* const weights =
      reinterpret_cast<float4*>(results + (kMove == kPlaces ? kRows * pitch : 0));
  const int group = threadIdx.x / threads, groups = kThreads / threads;
  const int t = threadIdx.x % threads, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const float share = 1.0f / (float)dim;
  const auto place = [&](int turn, int row, int which, int q) {
    return held + (((turn * kRows + row) * 2 + which) * pitch + q);
  };
  F2 w[kQuads][N], dw[kQuads][N], db[kQuads][N];
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int q = k * threads + t;
    load_vector<V, kWide>(in.w, q * V, dim - q * V, 1.0f, w[k]);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[k][i] = db[k][i] = 0;
    if (group != 0 || q >= quads) continue;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float4 v;
      unpack2(w[k][i], v.x, v.y);
      unpack2(w[k][i + 1], v.z, v.w);
      weights[i / 2 * quads + q] = v;
    }
  }
  const auto fetch = [&](int64_t r0, int turn) {
    if constexpr (kMove == kElements) {
      for (int i = group; i < kRows && r0 + i < in.rows; i += groups) {
        const T* px = in.x + row_offset(r0 + i, in.len, in.xs);
        const T* pg = dy + row_offset(r0 + i, in.len, ds);
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
          const int q = k * threads + t;
          if (q >= quads) continue;
          Q x, g;
          x.load(px + q * V, dim - q * V);
          g.load(pg + q * V, dim - q * V);
          *place(turn, i, 0, q) = x.q;
          *place(turn, i, 1, q) = g.q;
        }
      }
    }
    // a warp a row of x or of dy, or several warps one
    constexpr int kWarps = kThreads / 32, kShare = kWarps > 2 * kRows ? kWarps / (2 * kRows) : 1;
    const int first = warp % kShare * 32 + lane;
    for (int u = warp / kShare;
         kMove != kElements && u < 2 * kRows && r0 + u / 2 < in.rows; u += kWarps / kShare) {
      const int i = u / 2, which = u % 2;
      const T* p = which ? dy + row_offset(r0 + i, in.len, ds)
                         : in.x + row_offset(r0 + i, in.len, in.xs);
      uint4* to = place(turn, i, which, 0);
      if constexpr (kWide) {
#pragma unroll 2
        for (int q = first; q < quads; q += 32 * kShare) copy16(to + q, p + q * V);
      } else {
        if (first == 0) sh.shift[turn][i][which] = R::shift(p);
        R::fetch(to, p, dim, which ? dy : in.x, which ? dy_end : in.end, first, 32 * kShare);
      }
    }
    if (threadIdx.x < 3 * kRows && r0 + threadIdx.x / 3 < in.rows)
      copy4(&sh.stats[turn][0][0] + threadIdx.x, stats + 3 * r0 + threadIdx.x);
    copy_commit();
  };
  const auto row_quad = [&](int turn, int row, int which, int q) {
    Q r;
    if constexpr (kMove != kPlaces) r.q = *place(turn, row, which, q);
    else r.q = R::quad(place(turn, row, which, 0), q, sh.shift[turn][row][which], dim - q * V);
    return r;
  };
  const auto flush = [&](int64_t r0) {  // dx of a turn, with kPlaces
    const int i = warp / W;  // (as for its sums)
    if (r0 + i < in.rows)
      R::store(dx + row_offset(r0 + i, in.len, os), results + i * pitch, dim,
               warp % W * 32 + lane, 32 * W);
  };
  int64_t r0 = (int64_t)blockIdx.x * kRows;
  const int64_t step = (int64_t)gridDim.x * kRows;
  fetch(r0, 0);
  for (int turn = 0; r0 < in.rows; r0 += step, turn ^= 1) {
    copy_wait<0>();
    __syncthreads();  // (and all have done with the turn before)
    fetch(r0 + step, turn ^ 1);
    if (kMove == kPlaces && r0 >= step) flush(r0 - step);
    const int many = (int)min((int64_t)kRows, in.rows - r0);
    if (const int i = warp / W; i < many) {
      const float* st = sh.stats[turn][i];
      const F2 minus = pack2(-st[0], -st[0]), rstd = pack2(st[2], st[2]);
      const F2 shift = pack2(-st[1] * st[2], -st[1] * st[2]);
      F2 s1 = 0, s2 = 0;
#pragma unroll 2
      for (int q = warp % W * 32 + lane; q < quads; q += W * 32) {
        const Q x = row_quad(turn, i, 0, q), g = row_quad(turn, i, 1, q);
        // (behind the row dy is zero, and what n is there reaches nothing)
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const float4 v = weights[j / 2 * quads + q];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const F2 u = g.pair(j + e), c = e == 0 ? pack2(v.x, v.y) : pack2(v.z, v.w);
            const F2 n = fma2(add2(x.pair(j + e), minus), rstd, shift);
            s1 = fma2(u, c, s1);
            s2 = fma2(mul2(u, c), n, s2);
          }
        }
      }
      const float c = warp_sum2(both(s1), both(s2));
      if (lane % 16 == 0) sh.sums[i][lane / 16][warp % W] = c;
    }
    __syncthreads();
    for (int i = group; i < many; i += groups) {
      const float* st = sh.stats[turn][i];
      const F2 minus = pack2(-st[0], -st[0]), rstd = pack2(st[2], st[2]);
      const F2 shift = pack2(-st[1] * st[2], -st[1] * st[2]);
      float v1 = sh.sums[i][0][0], v2 = sh.sums[i][1][0];
#pragma unroll
      for (int k = 1; k < W; ++k) v1 += sh.sums[i][0][k], v2 += sh.sums[i][1][k];
      const float a1 = v1 * share * -st[2], a2 = v2 * share * -st[2];
      const F2 p1 = pack2(a1, a1), p2 = pack2(a2, a2);
      T* out = dx + row_offset(r0 + i, in.len, os);
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int q = k * threads + t;
        if (q >= quads) continue;
        const Q x = row_quad(turn, i, 0, q), g = row_quad(turn, i, 1, q);
        F2 o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const F2 u = g.pair(j);
          const F2 n = fma2(add2(x.pair(j), minus), rstd, shift);
          dw[k][j] = fma2(u, n, dw[k][j]);
          db[k][j] = add2(db[k][j], u);
          o[j] = fma2(n, p2, fma2(mul2(u, w[k][j]), rstd, p1));
        }
        if constexpr (kWide) *reinterpret_cast<uint4*>(out + q * V) = Q::packed(o);
        else if constexpr (kMove == kElements) Q::store(out + q * V, o, dim - q * V);
        else results[i * pitch + q] = Q::packed(o);
      }
    }
  }
  copy_wait<0>();
  if constexpr (kMove == kPlaces) {
    __syncthreads();
    flush(r0 - step);
  }
  if (part == nullptr) return;
  float* const out = part + (int64_t)blockIdx.x * 2 * dim;
  float* const sums = reinterpret_cast<float*>(shared);
  for (int g = 0; g < groups; ++g) {  // group by group, in order
    if (groups > 1) __syncthreads();
    if (group != g) continue;
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = (k * threads + t) * V + e;
        if (c >= dim) continue;
        float a[2], b[2];
        unpack2(dw[k][e / 2], a[0], a[1]);
        unpack2(db[k][e / 2], b[0], b[1]);
        if (groups == 1) {
          out[c] = a[e % 2];
          out[dim + c] = b[e % 2];
        } else {
          sums[c] = g == 0 ? a[e % 2] : sums[c] + a[e % 2];
          sums[dim + c] = g == 0 ? b[e % 2] : sums[dim + c] + b[e % 2];
        }
      }
  }
  if (groups == 1) return;
  __syncthreads();
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
#pragma unroll 4
  for (int64_t c = threadIdx.x; c < in.dim; c += kLongThreads) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float g = to_f32(d[c]) * (in.w != nullptr ? in.w[c] : 1.0f);
    s1 += g;
    s2 = fmaf(g, n, s2);
  }
  float v[2] = {s1, s2};
  row_sum(v, Team(kLongThreads), buf);
  const float a1 = v[0] / (float)in.dim, a2 = v[1] / (float)in.dim;
  T* o = dx + row_offset(r, in.len, os);
#pragma unroll 4
  for (int64_t c = threadIdx.x; c < in.dim; c += kLongThreads) {
    const float n = ((to_f32(x[c]) - st.mean) - st.rest) * st.rstd;
    const float g = to_f32(d[c]) * (in.w != nullptr ? in.w[c] : 1.0f);
    o[c] = from_f32<T>(st.rstd * fmaf(-n, a2, g - a1));
  }
}

// Rows of a partial sum of long rows. (4096 rows of 9001 in bf16 / of 6001 in fp32, us
// with 256: 311 / 312, 64: 207 / 199, 32: 211 / 176.)
constexpr int kSumRows = 64;

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

// Where a tensor of rows ends.
template <class T>
const T* rows_end(const cr_layer_norm_args* a, const void* p, Rows2 s) {
  if (a->batch == 0 || a->len == 0) return static_cast<const T*>(p);
  return static_cast<const T*>(p) + (a->batch - 1) * s.bs + (a->len - 1) * s.ts + a->dim;
}

template <class T>
NormIn<T> norm_in(const cr_layer_norm_args* a, bool one_batch) {
  return {a->batch * a->len, one_batch ? 0 : a->len, a->dim, a->eps, static_cast<const T*>(a->x),
          {a->x_batch_stride, a->x_time_stride}, a->weight, a->bias,
          rows_end<T>(a, a->x, {a->x_batch_stride, a->x_time_stride})};
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

// How a row lies in threads: by its length and type alone, so that its bits are
// the same among any others. (8 quads a lane before a second warp: with 4 rows of
// 4096 in bf16 took 94 us for 87, rows of 1024 in fp32 23 for 22.)
constexpr int kMostQuads = 8;
struct NormShape {
  int quads;    // 16 bytes a lane
  int threads;  // of a row, 0: more than registers hold
};
NormShape norm_shape(int64_t dim, size_t es) {
  const int64_t quads = ceil_div(dim, (int64_t)(16 / es));
  NormShape sh = {2, 32};
  while (sh.quads < kMostQuads && (int64_t)sh.quads * 32 < quads) sh.quads *= 2;
  while ((int64_t)sh.quads * sh.threads < quads) sh.threads *= 2;
  if (sh.threads > kNormThreads) sh.threads = 0;
  return sh;
}

// The backward call's: a block's threads, those of a row's columns, the rows of a
// turn, and blocks, which leave a part of the sums over rows each.
struct BackwardShape {
  int block, quads, threads, rows;
  int64_t blocks;  // 0: rows too long for it
};
BackwardShape backward_shape(int64_t rows, int64_t dim, size_t es) {
  const int64_t quads = ceil_div(dim, (int64_t)(16 / es));
  BackwardShape sh = {256, 1, 32, 4, 0};
  if (quads > 1024) return sh;
  if (quads > 256) sh.block = 512;
  if (quads > 512) sh.quads = 2, sh.rows = 2;
  if (quads <= 32) sh.rows = 8;  // (a warp a row)
  while ((int64_t)sh.quads * sh.threads < quads) sh.threads *= 2;
  sh.blocks = std::min<int64_t>(ceil_div(rows, sh.rows), 152 * (sh.block == 256 ? 2 : 1));
  return sh;
}

bool norm_wide(const cr_layer_norm_args* a) {
  const size_t es = model_esize(a->dt);
  return a->dim % (int64_t)(16 / es) == 0 &&
         rows_aligned(a->x, a->x_batch_stride, a->x_time_stride, es, 16) &&
         ptr_aligned(a->weight, 16) && ptr_aligned(a->bias, 16);
}

// Short rows are of fewer quads than this. Measured, 2^24 elements, us with elements
// / places, 16 bits forward: 30 quads 41 / 49, 45 39 / 41, 60 39 / 31, 120 50 / 33,
// 400 59 / 31 (32 bits: 45 / 62 at 45, 37 / 39 at 200, so elements alone); gradient:
// 65,536 rows of 333 (42 quads) 103 / 126, 16,384 of 2049 166 / 124, 32,768 of 777
// in 32 bits (195) 131 / 118.
constexpr int kShortQuads = 48;
template <class T>
Move norm_move(bool wide, int64_t dim, bool backward) {
  if (wide) return kWhole;
  return (backward || sizeof(T) == 2) && ceil_div(dim, (int64_t)(16 / sizeof(T))) >= kShortQuads
             ? kPlaces
             : kElements;
}

// Runs EXPR with the move M bound; PLACES, ELEMENTS: whether a call may have it.
#define CR_NORM_MOVE(MOVE, PLACES, ELEMENTS, ...)          \
  if ((MOVE) == kWhole) {                                  \
    constexpr Move M = kWhole;                             \
    __VA_ARGS__;                                           \
  } else if ((MOVE) == kPlaces) {                          \
    if constexpr (PLACES) {                                \
      constexpr Move M = kPlaces;                          \
      __VA_ARGS__;                                         \
    }                                                      \
  } else if constexpr (ELEMENTS) {                         \
    constexpr Move M = kElements;                          \
    __VA_ARGS__;                                           \
  }

template <class T, int Q>
bool launch_norm_quads(const NormIn<T>& in, int threads, T* y, Rows2 ys, float* stats, bool wide,
                       cudaStream_t s) {
  const int groups = kNormThreads / threads;
  const Move move = norm_move<T>(wide, in.dim, false);
  const size_t smem = (move == kPlaces ? norm_rows_bytes<Q, kPlaces>(groups)
                                       : norm_rows_bytes<Q, kWhole>(groups)) +
                      (y != nullptr ? (size_t)8 * Q * threads * (16 / sizeof(T)) : 0);
  // blocks an SM: as many as registers hold (65,536 rows of 768 in bf16, 4 quads: 39
  // us with 3, 45 with 4, 41 with 2; of 256, 2 quads: 23 with 3, 22 with 4, 23 with
  // 6; 16,384 rows of 1024 in fp32, 8 quads: 22 with 2, 27 with 4)
  constexpr int kFit = Q == 8 ? 2 : Q == 4 ? 3 : 4;
  const int64_t fit = std::min<int64_t>(kFit, (int64_t)(224 * 1024 / (smem + 2048)));
  const int64_t blocks = std::min(ceil_div(in.rows, kNormThreads / threads), 152 * fit);
  bool done = false;
  // (2 quads a lane: rows of up to 64 quads, others longer ones)
  CR_NORM_MOVE(move, sizeof(T) == 2, sizeof(T) == 4 || Q == 2,
               CR_LAUNCH(kKLayerNorm, s,
                         done = launch_clusters(layer_norm_kernel<T, Q, M>, blocks, 1,
                                                kNormThreads, smem, s, in, threads, y, ys,
                                                stats)))
  return done;
}

bool launch_norm(const cr_layer_norm_args* a, void* y, Rows2 ys, float* stats, bool wide,
                 cudaStream_t s) {
  const NormShape sh = norm_shape(a->dim, model_esize(a->dt));
  const Rows2 xs = {a->x_batch_stride, a->x_time_stride};
  const bool one = even(a->batch, a->len, xs) && even(a->batch, a->len, ys);
  bool done = true;
  CR_MODEL_TYPE(a->dt, {
    T* out = static_cast<T*>(y);
    const NormIn<T> in = norm_in<T>(a, one);
    if (sh.threads == 0)
      CR_LAUNCH(kKLayerNorm, s,
                layer_norm_long_kernel<T><<<(unsigned)in.rows, kLongThreads, 0, s>>>(in, out, ys,
                                                                                     stats));
    else if (sh.quads == 2) done = launch_norm_quads<T, 2>(in, sh.threads, out, ys, stats, wide, s);
    else if (sh.quads == 4) done = launch_norm_quads<T, 4>(in, sh.threads, out, ys, stats, wide, s);
    else done = launch_norm_quads<T, 8>(in, sh.threads, out, ys, stats, wide, s);
  });
  return done;
}

template <class T, int B, int Q, int R>
bool launch_norm_backward(const NormIn<T>& in, const BackwardShape& sh, const T* dy, Rows2 ds,
                          const T* dy_end, const float* stats, T* dx, Rows2 os, float* part,
                          bool wide, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const size_t quads = (size_t)ceil_div(in.dim, (int64_t)V);
  const Move move = norm_move<T>(wide, in.dim, true);
  const size_t smem = 16 * (move == kPlaces ? (quads + 1) * 5 * R : quads * 4 * R) + 4 * V * quads;
  bool done = false;
  // (8 rows a turn: rows of up to 32 quads; 512 threads: of more than 256)
  CR_NORM_MOVE(move, R != 8, B == 256,
               CR_LAUNCH(kKLayerNormBackward, s,
                         done = launch_clusters(layer_norm_backward_kernel<T, B, Q, R, M>,
                                                sh.blocks, 1, B, smem, s, in, sh.threads, dy, ds,
                                                dy_end, stats, dx, os, part)))
  return done;
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
  const bool done = launch_norm(a, y, ys, stats, wide, s);
  return done && cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

size_t cr_layer_norm_backward_workspace_bytes(int64_t batch, int64_t len, int64_t dim) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || (len > 0 && batch > kMaxBlocks / len)) return 0;
  const int64_t rows = batch * len;
  // (of the types' shapes the one with more parts)
  const int64_t parts = std::max({backward_shape(rows, dim, 2).blocks,
                                  backward_shape(rows, dim, 4).blocks,
                                  dim > 4096 ? ceil_div(rows, kSumRows) : (int64_t)0});
  return round256((size_t)rows * 12) + round256((size_t)parts * dim * 8) + kStatusBytes;
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
  const BackwardShape sh = backward_shape(rows, a->dim, es);
  const bool wide = norm_wide(a) &&
                    rows_aligned(g->dy, g->dy_batch_stride, g->dy_time_stride, es, 16) &&
                    rows_aligned(g->dx, g->dx_batch_stride, g->dx_time_stride, es, 16);
  const int64_t sum_blocks = ceil_div(2 * a->dim, 32), cols = ceil_div(a->dim, 256);
  if (sum_blocks > kMaxBlocks) return CR_ERR_UNSUPPORTED;
  char* at = past_status(ws);
  float* kept = reinterpret_cast<float*>(at);
  const bool sums = g->dweight != nullptr || g->dbias != nullptr;
  float* part = sums ? reinterpret_cast<float*>(at + round256((size_t)rows * 12)) : nullptr;
  const int64_t parts = sh.blocks != 0 ? sh.blocks : ceil_div(rows, kSumRows);
  const Rows2 xs = {a->x_batch_stride, a->x_time_stride};
  const float* stats = g->stats;
  bool done = true;
  if (rows > 0 && stats == nullptr) {
    done = launch_norm(a, nullptr, xs, kept, norm_wide(a), s);
    stats = kept;
  }
  const bool one = even(a->batch, a->len, xs) && even(a->batch, a->len, ds) &&
                   even(a->batch, a->len, os);
  CR_MODEL_TYPE(a->dt, {
    const T* dy = static_cast<const T*>(g->dy);
    T* dx = static_cast<T*>(g->dx);
    const NormIn<T> in = norm_in<T>(a, one);
    if (rows > 0 && sh.blocks == 0) {
      CR_LAUNCH(kKLayerNormBackward, s,
                layer_norm_backward_long_kernel<T><<<(unsigned)rows, kLongThreads, 0, s>>>(
                    in, dy, ds, stats, dx, os));
      if (sums)
        CR_LAUNCH(kKLayerNormSum, s,
                  layer_norm_part_kernel<T>
                  <<<dim3((unsigned)cols, (unsigned)std::min<int64_t>(parts, 65535)), 256, 0, s>>>(
                      in, dy, ds, stats, part));
    } else if (rows > 0) {
      const auto run = [&](auto launch) {
        return launch(in, sh, dy, ds, rows_end<T>(a, dy, ds), stats, dx, os, part, wide, s);
      };
      done = done && (sh.quads == 2     ? run(launch_norm_backward<T, 512, 2, 2>)
                      : sh.block == 512 ? run(launch_norm_backward<T, 512, 1, 4>)
                      : sh.rows == 4    ? run(launch_norm_backward<T, 256, 1, 4>)
                                        : run(launch_norm_backward<T, 256, 1, 8>));
    }
    if (sums)
      CR_LAUNCH(kKLayerNormSum, s,
                layer_norm_sum_kernel<<<(unsigned)sum_blocks, 1024, 0, s>>>(part, parts, a->dim,
                                                                            g->dweight, g->dbias));
  });
  return done && cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
