// Gated linear recurrence over time, its gradient, and its single-token form.
//
//   a[t] = sigmoid(gate[t]), r[t] = 1 - a[t] = sigmoid(-gate[t])
//   h[t] = a[t] h[t-1] + r[t] x[t],   y[t] = h[t] silu(z[t])
//   G[t] = dy[t] silu(z[t]) + a[t+1] G[t+1]
//   dx = r G,  dgate = (h[t-1] - x) G a r,  dz = dy h silu'(z)
//
// The state goes by r alone: where a memory is long, a is near 1 and binary32
// keeps few digits of r in it (a product by a would forget at a rate that is
// off by 2^-25 / r). So a h is h - r h, one rounding (of h, where little of it is
// left), exact for r = 0 and 1. An infinity becomes NaN in it, and NaN stays NaN: a
// sequence that ends in something not finite is gone through again, with products that
// keep infinities (kInf).
#include <algorithm>
#include <cfloat>
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
  const T* end;
};

template <class T>
struct GateIn {
  int64_t batch, len, dim;
  Strided<T> x, gate, z;
  const float* state;
  const void* lengths;
  int32_t index_bytes;
};

// C values that are worked on at once.
template <int C>
struct Vec;
template <>
struct Vec<1> {
  float v;
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ explicit Vec(float f) : v(f) {}
  __device__ __forceinline__ float get(int) const { return v; }
  __device__ __forceinline__ void set(int, float f) { v = f; }
};
template <>
struct Vec<2> {
  F2 v;
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ explicit Vec(float f) : v(pack2(f, f)) {}
  __device__ __forceinline__ Vec(float lo, float hi) : v(pack2(lo, hi)) {}
  __device__ __forceinline__ float get(int k) const {
    float lo, hi;
    unpack2(v, lo, hi);
    return k ? hi : lo;
  }
  __device__ __forceinline__ void set(int k, float f) {
    float lo, hi;
    unpack2(v, lo, hi);
    v = k ? pack2(lo, f) : pack2(f, hi);
  }
};
__device__ __forceinline__ Vec<1> fma(Vec<1> a, Vec<1> b, Vec<1> c) {
  return Vec<1>(fmaf(a.v, b.v, c.v));
}
__device__ __forceinline__ Vec<1> mul(Vec<1> a, Vec<1> b) { return Vec<1>(a.v * b.v); }
// not of a product (see add2)
__device__ __forceinline__ Vec<1> add(Vec<1> a, Vec<1> b) { return Vec<1>(a.v + b.v); }
__device__ __forceinline__ Vec<1> exp2_of(Vec<1> a) { return Vec<1>(exp2_fast(a.v)); }
__device__ __forceinline__ Vec<1> reciprocal_of(Vec<1> a) { return Vec<1>(reciprocal(a.v)); }
__device__ __forceinline__ Vec<2> fma(Vec<2> a, Vec<2> b, Vec<2> c) {
  Vec<2> r;
  r.v = fma2(a.v, b.v, c.v);
  return r;
}
__device__ __forceinline__ Vec<2> mul(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  r.v = mul2(a.v, b.v);
  return r;
}
__device__ __forceinline__ Vec<2> add(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  r.v = add2(a.v, b.v);
  return r;
}
__device__ __forceinline__ Vec<2> exp2_of(Vec<2> a) {
  return Vec<2>(exp2_fast(a.get(0)), exp2_fast(a.get(1)));
}
__device__ __forceinline__ Vec<2> reciprocal_of(Vec<2> a) {
  return Vec<2>(reciprocal(a.get(0)), reciprocal(a.get(1)));
}

// -1 / (1 + exp2(v s)), s = log2(e) or its negative. The product's rounding is
// |v| / 2 roundings of the result.
template <int C>
__device__ __forceinline__ Vec<C> minus_sigmoid(Vec<C> v, float s, Vec<C>* e_out = nullptr) {
  const Vec<C> e = exp2_of(mul(v, Vec<C>(s)));
  if (e_out != nullptr) *e_out = e;
  return reciprocal_of(fma(e, Vec<C>(-1.0f), Vec<C>(-1.0f)));
}

// An exponential that may be infinite, as the largest number.
template <int C>
__device__ __forceinline__ Vec<C> finite_of(Vec<C> e) {
  Vec<C> v;
#pragma unroll
  for (int k = 0; k < C; ++k) v.set(k, fminf(e.get(k), FLT_MAX));
  return v;
}

// A step for r: p - r p, and with what is added. kInf: what is infinite stays so (all
// else has the same bits).
template <bool kInf = false, int C>
__device__ __forceinline__ Vec<C> decay(Vec<C> minus_r, Vec<C> p) {
  Vec<C> v = fma(minus_r, p, p);
  if constexpr (kInf) {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (isinf(p.get(k)) && !isnan(minus_r.get(k))) v.set(k, p.get(k));
  }
  return v;
}
// Whether one of the channels that exist is infinite or NaN.
template <class V>
__device__ __forceinline__ bool odd(const V& v, int have) {
  return (have > 0 && !(fabsf(v[0]) < INFINITY)) ||
         (have > 1 && !(fabsf(v[sizeof(V) / 4 - 1]) < INFINITY));
}

// What a run of steps does to the state: h -> L + P h. Where P is near 1 its
// digits are in Q = 1 - P, where it is near 0 in P: kept is the smaller one, as Q or
// -P, so that a run is as exact as its steps.
template <int C>
struct alignas(8 * C) Map {
  float L[C], F[C];
  template <bool kInf>
  __device__ __forceinline__ void apply(float (&h)[C]) const {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const float v = fmaf(-F[k], h[k], L[k]);
      const float next = __float_as_int(F[k]) >= 0 ? v + h[k] : v;
      h[k] = kInf && isinf(h[k]) ? h[k] + L[k] : next;
    }
  }
};
template <int C>
__device__ __forceinline__ Map<C> run_map(Vec<C> L, Vec<C> minus_Q, Vec<C> P) {
  Map<C> m;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    m.L[k] = L.get(k);
    // (fabsf: the zero of a run that holds the state is not negative)
    m.F[k] = minus_Q.get(k) >= -0.5f ? fabsf(minus_Q.get(k)) : -P.get(k);
  }
  return m;
}
// The map b after the map a.
template <bool kInf, int C>
__device__ __forceinline__ Map<C> map_join(const Map<C>& a, const Map<C>& b) {
  Vec<C> L, q, p;
  float l[C];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const bool na = __float_as_int(a.F[k]) >= 0, nb = __float_as_int(b.F[k]) >= 0;
    const float Pa = na ? 1.0f - a.F[k] : -a.F[k], Pb = nb ? 1.0f - b.F[k] : -b.F[k];
    const float qa = na ? -a.F[k] : -a.F[k] - 1.0f, qb = nb ? -b.F[k] : -b.F[k] - 1.0f;  // P - 1
    q.set(k, fmaf(qb, Pa, qa));
    p.set(k, Pa * Pb);
    l[k] = a.L[k];
  }
  b.template apply<kInf>(l);
#pragma unroll
  for (int k = 0; k < C; ++k) L.set(k, l[k]);
  return run_map(L, q, p);
}

// A tile: 8 warps, each a run of kRun steps, a lane 32 bits of each step: one
// channel of binary32, two neighbours of 16 bits, which come by way of shared
// memory, 16 bytes an access, a tile ahead of their use (kWide: rows on 16 bytes;
// otherwise the places of 16 bytes that they lie in: 4 x 4096 x 2047 in bf16 takes
// 109 us, its gradient 198, where 2048 takes 61 and 105; by words of 4 bytes 179 and
// 334, read channel by channel 461 and 627).
constexpr int kRun = kGateCheckpoint;
constexpr int kGateWarps = 8;
constexpr int kTileSteps = kRun * kGateWarps;
constexpr int kMostCluster = 8;

template <class T>
struct Lane {
  static constexpr int C = 4 / sizeof(T);  // channels
};

template <class T, bool kWide>
struct Word {
  static constexpr int C = Lane<T>::C;
  static __device__ __forceinline__ Vec<C> get(uint32_t w) {
    if constexpr (sizeof(T) == 4) return Vec<C>(__uint_as_float(w));
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return Vec<C>(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
      return Vec<C>(f.x, f.y);
    }
  }
  static constexpr uint32_t kHeld =  // a gate of +infinity
      sizeof(T) == 4 ? 0x7F800000u : std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
  static __device__ __forceinline__ uint32_t round(Vec<C> f) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(f.get(0));
    else if constexpr (std::is_same<T, __half>::value) {
      const __half2 q = __floats2half2_rn(f.get(0), f.get(1));
      return *reinterpret_cast<const uint32_t*>(&q);
    } else {
      const __nv_bfloat162 q = __floats2bfloat162_rn(f.get(0), f.get(1));
      return *reinterpret_cast<const uint32_t*>(&q);
    }
  }
  static __device__ __forceinline__ void store(T* p, int have, uint32_t w) {
    if constexpr (sizeof(T) == 4 || kWide) {
      if (have > 0) *reinterpret_cast<uint32_t*>(p) = w;
    } else {
      unsigned short* q = reinterpret_cast<unsigned short*>(p);
      if (have > 1 && (uintptr_t)p % 4 == 0) {
        *reinterpret_cast<uint32_t*>(q) = w;
      } else {
        if (have > 0) q[0] = (unsigned short)w;
        if (have > 1) q[1] = (unsigned short)(w >> 16);
      }
    }
  }
};

// A run of one tensor in shared memory, a warp's own: kRun rows of 128 bytes, or
// of the places of 16 bytes that these lie in.
template <bool kWide>
struct Staged {
  uint32_t w[kRun][kWide ? 32 : 36];
};

// One input's runs, by way of shared memory. Steps past the end read as `past`
// (two channels of it).
template <class T, bool kWide>
struct Runs {
  static constexpr int E = 16 / sizeof(T);  // elements of an access, which divide dim
  Staged<kWide>* staged;
  const T* p;  // this lane's first access of step 0
  int64_t ts;
  bool have;
  uint32_t past;
  __device__ __forceinline__ Runs(const Strided<T>& s, int64_t b, int64_t group, int64_t dim,
                                  Staged<kWide>* st, uint32_t past_ = 0u)
      : staged(st), ts(s.ts), past(past_) {
    const int lane = threadIdx.x % 32;
    const int64_t c = group * 32 * Lane<T>::C + lane % 8 * E;
    have = c < dim;
    p = s.p + b * s.bs + (have ? c : 0) + lane / 8 * ts;
  }
  // begins to fetch steps t0 .. t0 + m
  __device__ __forceinline__ void ask(int64_t t0, int m) const {
    const int lane = threadIdx.x % 32;
    const T* from = p + t0 * ts;
    uint32_t* to = &staged->w[lane / 8][lane % 8 * 4];
    if (m == kRun) {
#pragma unroll
      for (int j = 0; j < kRun / 4; ++j)
        if (have) copy16(to + j * 128, from + j * 4 * ts);
    } else {
#pragma unroll
      for (int j = 0; j < kRun / 4; ++j) {
        if (j * 4 + lane / 8 >= m)
          *reinterpret_cast<uint4*>(to + j * 128) = make_uint4(past, past, past, past);
        else if (have)
          copy16(to + j * 128, from + j * 4 * ts);
      }
    }
  }
  __device__ __forceinline__ uint32_t get(int i) const { return staged->w[i][threadIdx.x % 32]; }
};

// Rows that start anywhere lie in shared memory as they do in their places, some
// elements off, and are put right as they are taken. What is beside the row in its
// first and last place is read where the tensor has it, and left out.
template <class T>
struct Runs<T, false> {
  static constexpr int kHalves = Lane<T>::C, E = 16 / sizeof(T), kChannels = 32 * kHalves;
  const Strided<T>& s;
  Staged<false>* staged;
  const T* p;      // the group's first channel of step 0
  int left;        // channels from there on
  int first, more;  // elements that step 0 is off its place, and a step from the one before
  uint32_t past;
  __device__ __forceinline__ Runs(const Strided<T>& s_, int64_t b, int64_t group, int64_t dim,
                                  Staged<false>* st, uint32_t past_ = 0u)
      : s(s_), staged(st), past(past_) {
    const int64_t c = group * kChannels;
    p = s.p + b * s.bs + c;
    left = (int)min((int64_t)(kChannels + E), dim - c);
    first = shift(p);
    more = (int)(s.ts % E);
  }
  static __device__ __forceinline__ int shift(const T* q) {
    return (int)((uintptr_t)q % 16) / (int)sizeof(T);
  }
  // Place `q` of the row at r.
  __device__ __forceinline__ void place(uint32_t* to, const T* r, int q) const {
    const int e = q * E - shift(r);
    if (e >= min(left, kChannels)) return;
    const T* const from = r + e;
    if ((e >= 0 && e + E <= left) || (from >= s.p && from + E <= s.end)) {
      copy16(to, from);
    } else {
      Pack<T, E> v;
#pragma unroll
      for (int i = 0; i < E; ++i)
        v.v[i] = e + i >= 0 && e + i < left ? from[i] : from_f32<T>(0.0f);
      *reinterpret_cast<uint4*>(to) = __builtin_bit_cast(uint4, v);
    }
  }
  __device__ __forceinline__ void ask(int64_t t0, int m) const {
    const int lane = threadIdx.x % 32;
    const T* const from = p + t0 * s.ts;
    const uint4 none = make_uint4(past, past, past, past);
#pragma unroll
    for (int j = 0; j < kRun / 4; ++j) {
      const int i = j * 4 + lane / 8;
      uint32_t* to = &staged->w[i][lane % 8 * 4];
      if (i < m) place(to, from + i * s.ts, lane % 8);
      else *reinterpret_cast<uint4*>(to) = none;
    }
    if (lane < kRun) {  // the ninth places
      uint32_t* to = &staged->w[lane][32];
      if (lane < m) place(to, from + lane * s.ts, 8);
      else *reinterpret_cast<uint4*>(to) = none;
    }
  }
  __device__ __forceinline__ uint32_t get(int i) const {
    // (runs begin at steps that are multiples of 16)
    int off = first;
    asm volatile("" : "+r"(off));  // (not all of a run's held in registers between turns)
    off = (off + i * more) & (E - 1);
    const uint32_t* w = &staged->w[i][threadIdx.x % 32 + off / kHalves];
    if constexpr (kHalves == 1) return *w;
    else return __funnelshift_r(w[0], w[1], off % 2 * 16);
  }
};

// Which channels a lane has.
template <class T>
struct Channels {
  static constexpr int C = Lane<T>::C;
  int64_t d;
  int have;
  __device__ Channels(int64_t group, int64_t dim) {
    d = (group * 32 + threadIdx.x % 32) * C;
    have = (int)max((int64_t)0, min((int64_t)C, dim - d));
    if (have == 0) d = 0;
  }
  __device__ __forceinline__ int64_t at(int k) const { return d + k; }
};

// The maps of a tile's warps and of a cluster's tiles, for this turn and the
// one before, which another block of the cluster may still be reading.
template <int C>
struct Joints {
  Map<C> warp[2][kGateWarps][32];
  Map<C> tile[2][kMostCluster][32];
};

// Gives the state that this warp's run starts from, and moves `carry` past all
// of the cluster's tiles. (Its first call comes after cluster_wait(): it writes to
// the other blocks' shared memory.)
template <int C, bool kBack, bool kInf>
__device__ __forceinline__ Vec<C> join_runs(Joints<C>& j, int turn, int rank, int blocks,
                                            const Map<C>& run, float (&carry)[C]) {
  namespace cg = cooperative_groups;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  j.warp[turn][warp][lane] = run;
  __syncthreads();
  float h[C];
#pragma unroll
  for (int k = 0; k < C; ++k) h[k] = carry[k];
  if (blocks > 1) {
    const cg::cluster_group cl = cg::this_cluster();
    // the tile's map, to every block of the cluster: warp w tells block w
    static_assert(kMostCluster <= kGateWarps, "a warp a block");
    if (warp < blocks) {
      Map<C> tile = j.warp[turn][kBack ? kGateWarps - 1 : 0][lane];
#pragma unroll 1  // (unrolled: one long prompt 131 us for 135, training 255 for 250)
      for (int i = 1; i < kGateWarps; ++i)
        tile = map_join<kInf>(tile, j.warp[turn][kBack ? kGateWarps - 1 - i : i][lane]);
      *cl.map_shared_rank(&j.tile[turn][rank][lane], warp) = tile;
    }
    cl.sync();
    for (int i = 0; i < blocks; ++i) {
      const int r = kBack ? blocks - 1 - i : i;
#pragma unroll
      for (int k = 0; k < C; ++k) h[k] = r == rank ? carry[k] : h[k];
      j.tile[turn][r][lane].template apply<kInf>(carry);
    }
#pragma unroll
    for (int i = 0; i < kGateWarps; ++i) {
      const int w = kBack ? kGateWarps - 1 - i : i;
      if (kBack ? w > warp : w < warp) j.warp[turn][w][lane].template apply<kInf>(h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGateWarps; ++i) {
      const int w = kBack ? kGateWarps - 1 - i : i;
#pragma unroll
      for (int k = 0; k < C; ++k) h[k] = w == warp ? carry[k] : h[k];
      j.warp[turn][w][lane].template apply<kInf>(carry);
    }
  }
  Vec<C> v;
#pragma unroll
  for (int k = 0; k < C; ++k) v.set(k, h[k]);
  return v;
}

template <class T>
struct GateFwd {
  T* y;
  int64_t ybs, yts;
  float* final_state;
  float* checkpoints;
  int64_t n_check;
};

template <int C, bool kWide>
struct ForwardShared {
  Joints<C> joints;
  Staged<kWide> staged[kGateWarps][3];
};

template <class T, bool kZ, bool kWide>
__global__ void __launch_bounds__(kGateWarps * 32, 2)
gated_scan_kernel(GateIn<T> in, GateFwd<T> out, int blocks) {
  constexpr int C = Lane<T>::C;
  using W = Word<T, kWide>;
  using V = Vec<C>;
  extern __shared__ __align__(16) char shared[];
  ForwardShared<C, kWide>& sh = *reinterpret_cast<ForwardShared<C, kWide>*>(shared);
  if (blocks > 1) cluster_arrive();
  const int warp = threadIdx.x / 32;
  const int rank = (int)(blockIdx.x % (unsigned)blocks);
  const int64_t per = (in.dim + 32 * C - 1) / (32 * C);
  int64_t group;
  const int64_t b = divide(blockIdx.x / (unsigned)blocks, per, group);
  const Channels<T> ch(group, in.dim);
  const int64_t n = sequence_length(in.lengths, in.index_bytes, b, in.len);
  Staged<kWide>* st = sh.staged[warp];
  const Runs<T, kWide> rg(in.gate, b, group, in.dim, st, W::kHeld);
  const Runs<T, kWide> rx(in.x, b, group, in.dim, st + 1);
  const Runs<T, kWide> rz(kZ ? in.z : in.x, b, group, in.dim, st + 2);
  float carry[C];  // -h
  const auto begin = [&] {
#pragma unroll
    for (int k = 0; k < C; ++k)
      carry[k] = in.state != nullptr && k < ch.have ? -in.state[b * in.dim + ch.at(k)] : 0.0f;
  };
  begin();
  const int64_t step = (int64_t)blocks * kTileSteps;
  // all of it, from the beginning (begun: what is waited for after the first loads)
  const auto turns = [&](auto inf, auto begun) {
    int turn = 0;
    int64_t t0 = (int64_t)rank * kTileSteps + warp * kRun;  // this warp's run
    auto steps = [&](int64_t t) { return (int)max((int64_t)0, min((int64_t)kRun, n - t)); };
    int m = steps(t0);
    rg.ask(t0, m);
    rx.ask(t0, m);
    copy_commit();
    if constexpr (kZ) rz.ask(t0, m);
    copy_commit();
    begun();
    for (int64_t s0 = 0; s0 < n; s0 += step, t0 += step, turn ^= 1) {
      uint32_t g[kRun], xw[kRun];
      copy_wait<1>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kRun; ++i) g[i] = rg.get(i);
#pragma unroll
      for (int i = 0; i < kRun; ++i) xw[i] = rx.get(i);
      __syncwarp();
      const int64_t next = t0 + step;
      const int m_next = steps(next);
      rg.ask(next, m_next);
      rx.ask(next, m_next);
      copy_commit();
      V r[kRun], x[kRun];  // -r
      V L(0.0f), Q(0.0f), P(1.0f);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        r[i] = minus_sigmoid(W::get(g[i]), kLog2e);
        x[i] = W::get(xw[i]);
        L = fma(r[i], x[i], decay<inf>(r[i], L));  // of the negative state
        Q = fma(r[i], P, Q);
        P = decay(r[i], P);
      }
      V s = join_runs<C, false, inf>(sh.joints, turn, rank, blocks, run_map(L, Q, P), carry);
      if (out.checkpoints != nullptr && m > 0) {
        float* p = out.checkpoints + (b * out.n_check + t0 / kRun) * in.dim;
#pragma unroll
        for (int k = 0; k < C; ++k)
          if (k < ch.have) p[ch.at(k)] = -s.get(k);
      }
      if constexpr (kZ) {
        copy_wait<1>();
        __syncwarp();
      }
      uint32_t y[kRun];
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        s = fma(r[i], x[i], decay<inf>(r[i], s));
        if constexpr (kZ) {
          const V z = W::get(rz.get(i));
          y[i] = W::round(mul(mul(s, z), minus_sigmoid(z, -kLog2e)));
        } else {
          y[i] = W::round(mul(s, V(-1.0f)));
        }
      }
      if constexpr (kZ) {
        __syncwarp();
        rz.ask(next, m_next);
      }
      copy_commit();
      T* py = out.y + b * out.ybs + t0 * out.yts + ch.d;
      if (m == kRun) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) W::store(py + i * out.yts, ch.have, y[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (i < m) W::store(py + i * out.yts, ch.have, y[i]);
      }
      m = m_next;
    }
    copy_wait<0>();
  };
  turns(std::false_type{}, [&] { if (blocks > 1) cluster_wait(); });
  // past the sequence's end
  for (int64_t t = n + rank * kGateWarps + warp; t < in.len; t += blocks * kGateWarps)
    W::store(out.y + b * out.ybs + t * out.yts + ch.d, ch.have, 0u);
  if (blocks > 1) cooperative_groups::this_cluster().sync();  // others write here
  if (__any_sync(~0u, odd(carry, ch.have))) {  // (the same in all of the cluster's warps)
    if (blocks == 1) __syncthreads();
    begin();
    turns(std::true_type{}, [] {});
    if (blocks > 1) cooperative_groups::this_cluster().sync();
  }
  if (out.final_state != nullptr && rank == 0 && warp == 0) {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (k < ch.have) out.final_state[b * in.dim + ch.at(k)] = -carry[k];
  }
}

template <class T>
struct GateOut {
  T *dx, *dgate, *dz;  // contiguous
  float* dstate;
};

template <int C, bool kWide>
struct BackwardShared {
  Joints<C> joints;
  Staged<kWide> staged[kGateWarps][4];
  int odd, any;  // whether a run's states are not all finite, of this block and of all
};

template <class T>
struct GateGrads {
  Strided<T> dy;
  const float *dfinal, *checkpoints;
  int64_t n_check;
  GateOut<T> out;
};

// The same again, with infinities kept, where something in a sequence is not finite:
// channel after channel of a lane, straight from memory, step after step of a run in
// shared memory. (Few registers: with a second loop like the kernel's, or a call of
// one, that one's spilled, and the gradient of 4 x 4096 x 4096 in bf16 took 172 to 220
// us for 160. Where this runs for all of it, that takes 1080; the forward pass, which
// has a second loop, 192 for 100.)
template <class T, bool kZ, bool kWide>
__device__ __forceinline__ void backward_again(const GateIn<T>& in, const GateGrads<T>& grads,
                                               int rank, int blocks, int64_t b, int64_t n,
                                               const Channels<T>& ch, Joints<1>& joints,
                                               Staged<kWide> (*staged)[4]) {
  using V = Vec<1>;
  constexpr int C = Lane<T>::C;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t step = (int64_t)blocks * kTileSteps;
  const auto held = [&](int which, int i) -> float& {
    return reinterpret_cast<float&>(staged[warp][which].w[i][lane]);
  };
#pragma unroll 1
  for (int k = 0; k < C; ++k) {
    const bool have = k < ch.have;
    const int64_t c = have ? ch.at(k) : 0;  // (lanes without one go through the first)
    float carry[1] = {grads.dfinal != nullptr && have ? -grads.dfinal[b * in.dim + c] : 0.0f};
    int turn = 0;
#pragma unroll 1
    for (int64_t s0 = (n + step - 1) / step * step - step; s0 >= 0; s0 -= step, turn ^= 1) {
      const int64_t t0 = s0 + rank * kTileSteps + warp * kRun;
      const int m = (int)max((int64_t)0, min((int64_t)kRun, n - t0));
      const auto read = [&](const Strided<T>& p, int i) {
        return V(to_f32(p.p[b * p.bs + (t0 + i) * p.ts + c]));
      };
      const int64_t at = (b * in.len + t0) * in.dim + c;
      V s(m > 0 ? -grads.checkpoints[(b * grads.n_check + t0 / kRun) * in.dim + c] : 0.0f);
#pragma unroll 2
      for (int i = 0; i < m; ++i) {
        const V x = read(in.x, i), g = read(in.gate, i);
        V e, v = read(grads.dy, i);
        const V r = minus_sigmoid(g, kLog2e, &e);
        held(0, i) = r.v;
        held(1, i) = mul(mul(add(s, x), r), mul(finite_of(e), r)).v;
        s = fma(r, x, decay<true>(r, s));
        if constexpr (kZ) {
          const V z = read(in.z, i), w = minus_sigmoid(z, -kLog2e);
          const V silu = mul(z, w), slope = fma(silu, fma(w, V(1.0f), V(1.0f)), w);
          if (have) grads.out.dz[at + i * in.dim] = from_f32<T>(mul(mul(v, s), slope).v);
          v = mul(v, silu);
        } else {
          v = mul(v, V(-1.0f));
        }
        held(2, i) = v.v;
      }
      V L(0.0f), Q(0.0f), P(1.0f);
#pragma unroll 1
      for (int i = m - 1; i >= 0; --i) {
        const V r(held(0, i));
        L = decay<true>(r, fma(V(held(2, i)), V(1.0f), L));
        Q = fma(r, P, Q);
        P = decay(r, P);
      }
      V B = join_runs<1, true, true>(joints, turn, rank, blocks, run_map(L, Q, P), carry);
#pragma unroll 1
      for (int i = m - 1; i >= 0; --i) {
        const V r(held(0, i)), G = fma(V(held(2, i)), V(1.0f), B);
        if (have) {
          grads.out.dx[at + i * in.dim] = from_f32<T>(mul(r, G).v);
          grads.out.dgate[at + i * in.dim] = from_f32<T>(mul(V(held(1, i)), G).v);
        }
        B = decay<true>(r, G);
      }
    }
    if (grads.out.dstate != nullptr && have && rank == 0 && warp == 0)
      grads.out.dstate[b * in.dim + c] = -carry[0];
    if (blocks > 1) cooperative_groups::this_cluster().sync();
    else __syncthreads();
  }
}

template <class T, bool kZ, bool kWide>
__global__ void __launch_bounds__(kGateWarps * 32, 2)
gated_scan_backward_kernel(const __grid_constant__ GateIn<T> in,
                           const __grid_constant__ GateGrads<T> grads, int blocks) {
  const Strided<T>& dy = grads.dy;
  const GateOut<T>& out = grads.out;
  const float* __restrict__ const dfinal = grads.dfinal;
  const float* __restrict__ const checkpoints = grads.checkpoints;
  constexpr int C = Lane<T>::C;
  using W = Word<T, kWide>;
  using V = Vec<C>;
  extern __shared__ __align__(16) char shared[];
  BackwardShared<C, kWide>& sh = *reinterpret_cast<BackwardShared<C, kWide>*>(shared);
  if (threadIdx.x == 0) sh.odd = sh.any = 0;
  if (blocks > 1) cluster_arrive();
  else __syncthreads();
  const int warp = threadIdx.x / 32;
  const int rank = (int)(blockIdx.x % (unsigned)blocks);
  const int64_t per = (in.dim + 32 * C - 1) / (32 * C);
  int64_t group;
  const int64_t b = divide(blockIdx.x / (unsigned)blocks, per, group);
  const Channels<T> ch(group, in.dim);
  const int64_t n = sequence_length(in.lengths, in.index_bytes, b, in.len);
  Staged<kWide>* st = sh.staged[warp];
  const Runs<T, kWide> rg(in.gate, b, group, in.dim, st, W::kHeld);
  const Runs<T, kWide> rx(in.x, b, group, in.dim, st + 1);
  const Runs<T, kWide> re(dy, b, group, in.dim, st + 2);
  const Runs<T, kWide> rz(kZ ? in.z : in.x, b, group, in.dim, st + 3);
  float carry[C];  // -a[t+1] G[t+1]
#pragma unroll
  for (int k = 0; k < C; ++k)
    carry[k] = dfinal != nullptr && k < ch.have ? -dfinal[b * in.dim + ch.at(k)] : 0.0f;
  const int64_t step = (int64_t)blocks * kTileSteps;
  int turn = 0;
  int64_t s0 = (n + step - 1) / step * step - step;
  auto steps = [&](int64_t t) {
    return t < 0 ? 0 : (int)max((int64_t)0, min((int64_t)kRun, n - t));
  };
  const int64_t mine = (int64_t)rank * kTileSteps + warp * kRun;
  int m = s0 < 0 ? 0 : steps(s0 + mine);
  float h[C];
  auto ask = [&](int64_t t0, int m) {
    rg.ask(t0, m);
    rx.ask(t0, m);
    re.ask(t0, m);
    if constexpr (kZ) rz.ask(t0, m);
    copy_commit();
    const float* p = checkpoints + (b * grads.n_check + t0 / kRun) * in.dim;
#pragma unroll
    for (int k = 0; k < C; ++k) h[k] = m > 0 && k < ch.have ? p[ch.at(k)] : 0.0f;
  };
  ask(s0 + mine, m);
  if (blocks > 1) cluster_wait();
  for (; s0 >= 0; s0 -= step, turn ^= 1) {
    const int64_t t0 = s0 + mine;
    const int64_t at = (b * in.len + t0) * in.dim + ch.d;
    copy_wait<0>();
    __syncwarp();
    // the states again; what the way back takes of each step, which goes by -G
    V r[kRun], d[kRun], v[kRun];  // -r, (x - h[t-1]) a r, -dy silu(z)
    V s;
#pragma unroll
    for (int k = 0; k < C; ++k) s.set(k, -h[k]);
    V Q(0.0f), P(1.0f);
    uint32_t dz[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const V x = W::get(rx.get(i));
      V e;
      r[i] = minus_sigmoid(W::get(rg.get(i)), kLog2e, &e);
      // e r = a keeps its digits where r is near 1 (and is 0 with r)
      d[i] = mul(mul(add(s, x), r[i]), mul(finite_of(e), r[i]));
      s = fma(r[i], x, decay(r[i], s));
      v[i] = W::get(re.get(i));
      if constexpr (kZ) {
        const V z = W::get(rz.get(i)), w = minus_sigmoid(z, -kLog2e);  // -sigmoid
        const V silu = mul(z, w);                                            // -silu
        // minus the slope: w + silu (1 + w), silu' = sigmoid + silu (1 - sigmoid)
        const V slope = fma(silu, fma(w, V(1.0f), V(1.0f)), w);
        dz[i] = W::round(mul(mul(v[i], s), slope));
        v[i] = mul(v[i], silu);
      } else {
        v[i] = mul(v[i], V(-1.0f));
      }
    }
    float last[C];
#pragma unroll
    for (int k = 0; k < C; ++k) last[k] = s.get(k);
    if (odd(last, ch.have)) sh.odd = 1;
    if constexpr (kZ) {
      if (m == kRun) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) W::store(out.dz + at + i * in.dim, ch.have, dz[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (i < m) W::store(out.dz + at + i * in.dim, ch.have, dz[i]);
      }
    }
    __syncwarp();
    const int64_t next = s0 - step;
    const int m_next = next < 0 ? 0 : steps(next + mine);
    ask(next < 0 ? t0 : next + mine, m_next);
    V L(0.0f);
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i) {
      L = decay(r[i], fma(v[i], V(1.0f), L));  // (a sum with a product: see add2)
      Q = fma(r[i], P, Q);
      P = decay(r[i], P);
    }
    V B = join_runs<C, true, false>(sh.joints, turn, rank, blocks, run_map(L, Q, P), carry);
    uint32_t ox[kRun], og[kRun];
#pragma unroll
    for (int i = kRun - 1; i >= 0; --i) {
      const V G = fma(v[i], V(1.0f), B);
      ox[i] = W::round(mul(r[i], G));
      og[i] = W::round(mul(d[i], G));
      B = decay(r[i], G);
    }
    if (m == kRun) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        W::store(out.dx + at + i * in.dim, ch.have, ox[i]);
        W::store(out.dgate + at + i * in.dim, ch.have, og[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (i < m) {
          W::store(out.dx + at + i * in.dim, ch.have, ox[i]);
          W::store(out.dgate + at + i * in.dim, ch.have, og[i]);
        }
      }
    }
    m = m_next;
  }
  copy_wait<0>();
  if (out.dstate != nullptr && rank == 0 && warp == 0) {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (k < ch.have) out.dstate[b * in.dim + ch.at(k)] = -carry[k];
  }
  for (int64_t t = n + rank * kGateWarps + warp; t < in.len; t += blocks * kGateWarps) {
    const int64_t at = (b * in.len + t) * in.dim + ch.d;
    W::store(out.dx + at, ch.have, 0u);
    W::store(out.dgate + at, ch.have, 0u);
    if constexpr (kZ) W::store(out.dz + at, ch.have, 0u);
  }
  __syncthreads();
  if (blocks > 1) {
    if (sh.odd && threadIdx.x < blocks)
      *cooperative_groups::this_cluster().map_shared_rank(&sh.any, threadIdx.x) = 1;
    cooperative_groups::this_cluster().sync();
  }
  // (the same in all of the cluster's warps)
  if (__any_sync(~0u, odd(carry, ch.have)) || (blocks > 1 ? sh.any : sh.odd))
    backward_again<T, kZ>(in, grads, rank, blocks, b, n, ch,
                          reinterpret_cast<Joints<1>&>(sh.joints), sh.staged);
}

// One token of each stream: a thread a channel, blocks of a stream side by side,
// so that all the state's reads are in flight at once. (64 streams of 4096 in bf16
// take 4.6 us, most of it the call's own; the bytes are 0.6.)
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
      const float r = minus_sigmoid(Vec<1>(to_f32(in.gate.p[b * in.gate.bs + d])), kLog2e).v;
      h = fmaf(-r, x, isinf(h) ? h : fmaf(r, h, h));
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
Strided<T> strided(const cr_gated_scan_args* a, const void* p, int64_t bs, int64_t ts) {
  const T* q = static_cast<const T*>(p);
  if (q == nullptr || a->batch == 0 || a->len == 0) return {q, bs, ts, q};
  return {q, bs, ts, q + (a->batch - 1) * bs + (a->len - 1) * ts + a->dim};
}

template <class T>
GateIn<T> gate_in(const cr_gated_scan_args* a) {
  return {a->batch, a->len, a->dim,
          strided<T>(a, a->x, a->x_batch_stride, a->x_time_stride),
          strided<T>(a, a->gate, a->gate_batch_stride, a->gate_time_stride),
          strided<T>(a, a->z, a->z_batch_stride, a->z_time_stride),
          a->state, a->lengths, a->index_bytes};
}

// Blocks that share a sequence's time: as many as fit the GPU at once with those
// of the other sequences and channels (two an SM). Each turn then waits for all of
// them, which few sequences repay and many do not. Measured, bf16, us for 1 / 2 / 4
// / 8 blocks: one sequence of 32,768 x 2048 481 / 300 / 156 / 135, 4 of 4096 x 4096
// with their gradient 250 / 305 / 297 / 346, 9 ragged ones to 517 x 1000 in fp16 14
// / 14 / 18 / 29.
int gate_blocks(int64_t groups, int64_t len) {
  const int64_t c = std::min(304 / groups, ceil_div(len, kTileSteps));
  return (int)std::max<int64_t>(1, std::min<int64_t>(c, kMostCluster));
}

// The kernel for a call with z or without, and for rows on 16 bytes or anywhere.
#define CR_GATE_KERNEL(NAME, T, Z, WIDE)             \
  (Z ? WIDE ? NAME<T, true, true> : NAME<T, true, false> \
     : WIDE ? NAME<T, false, true> : NAME<T, false, false>)

// Whether rows are on 16 bytes and whole accesses long.
bool gate_wide(const cr_gated_scan_args* a) {
  const size_t es = model_esize(a->dt);
  return a->dim % (int64_t)(16 / es) == 0 &&
         rows_aligned(a->x, a->x_batch_stride, a->x_time_stride, es, 16) &&
         rows_aligned(a->gate, a->gate_batch_stride, a->gate_time_stride, es, 16) &&
         (a->z == nullptr || rows_aligned(a->z, a->z_batch_stride, a->z_time_stride, es, 16));
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
  bool done = false;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    const GateFwd<T> out = {static_cast<T*>(y), y_batch_stride, y_time_stride, final_state,
                            checkpoints, cr_gated_scan_checkpoints(a->len)};
    const bool wide = gate_wide(a) && rows_aligned(y, y_batch_stride, y_time_stride, es, 4);
    const size_t smem = wide ? sizeof(ForwardShared<Lane<T>::C, true>)
                             : sizeof(ForwardShared<Lane<T>::C, false>);
    auto kernel = CR_GATE_KERNEL(gated_scan_kernel, T, (a->z != nullptr), wide);
    CR_LAUNCH(kKGatedScan, s,
              done = launch_clusters(kernel, a->batch * per * c, c, kGateWarps * 32, smem, s,
                                     gate_in<T>(a), out, c));
  });
  return done && cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
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
  bool done = false;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    const GateGrads<T> grads = {strided<T>(a, g->dy, g->dy_batch_stride, g->dy_time_stride),
                                g->dfinal, g->checkpoints, cr_gated_scan_checkpoints(a->len),
                                {static_cast<T*>(g->dx), static_cast<T*>(g->dgate),
                                 static_cast<T*>(g->dz), g->dstate}};
    const bool wide = gate_wide(a) &&
                      rows_aligned(g->dy, g->dy_batch_stride, g->dy_time_stride, es, 16) &&
                      ptr_aligned(g->dx, 4) && ptr_aligned(g->dgate, 4) && ptr_aligned(g->dz, 4);
    const size_t smem = wide ? sizeof(BackwardShared<Lane<T>::C, true>)
                             : sizeof(BackwardShared<Lane<T>::C, false>);
    auto kernel = CR_GATE_KERNEL(gated_scan_backward_kernel, T, (a->z != nullptr), wide);
    CR_LAUNCH(kKGatedScanBackward, s,
              done = launch_clusters(kernel, a->batch * per * c, c, kGateWarps * 32, smem, s,
                                     gate_in<T>(a), grads, c));
  });
  return done && cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
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
