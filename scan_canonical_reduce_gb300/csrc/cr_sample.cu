// The next token of each row of logits: temperature, top-k, top-p, min-p.
//
// The row's tokens in the order of falling logits (equal ones by index) are
// kept up to a border, and the token is where the running sum of their weights
// w = 2^-y, y = (largest - logit) log2(e) / temperature, exceeds u times the
// kept sum. So each limit is a border in one order, and each is found the same
// way: a histogram of y with 16 bins an octave, whose bins hold numbers and
// sums of weights, gives the bin; the bin's few tokens, gathered and sorted,
// give the place in it. (A bin of more tokens than can be sorted is cut again by
// the logits' bits, and one logit's tokens by their index.) Sums are of
// integers, so that no order of summation changes them, and are exact to 2^-32
// of a weight: the token is the one that exact arithmetic gives, unless a setting lies
// that near to a border.
//
// A row is one cluster of blocks, a slice each, held in shared memory where it
// fits. The first block leads: it has the row's sums and the list of a bin.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cooperative_groups.h>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kBins = 1024;   // 16 an octave
constexpr int kList = 1024;   // most tokens that are sorted
constexpr int kRanked = 128;  // up to so many by their ranks
constexpr int kFew = 512;     // top_k up to which its tokens alone are looked at
constexpr int kMostBlocks = 8;
constexpr int kMostSlice = 1 << 17;  // tokens of a block
constexpr uint32_t kOverflow = 2 * kMostSlice;
constexpr uint32_t kNone = 0xFFFFFFFFu;  // the key of what is no candidate
static_assert(kBins % kThreads == 0 && kList % kThreads == 0 && kBins % 1024 == 0,
              "a thread's bins and tokens, a lane's words of chosen bins");
static_assert(kBins % kMostBlocks == 0 && kRanked <= kThreads, "a block's bins, a token a thread");

// 2^(-j / 16) in units of 2^-63
__constant__ unsigned long long kRoots[16] = {
    0x8000000000000000ULL, 0x7A92BE8A92436616ULL, 0x75606373EE921C97ULL, 0x70666F76154A7089ULL,
    0x6BA27E656B4EB57AULL, 0x6712460A8FC24072ULL, 0x62B39508AA836D6FULL, 0x5E8451CFAC061B5FULL,
    0x5A827999FCEF3242ULL, 0x56AC1F752150A563ULL, 0x52FF6B54D8A89C75ULL, 0x4F7A993048D088D7ULL,
    0x4C1BF828C6DC54B8ULL, 0x48E1E9B9D588E19BULL, 0x45CAE0F1F545EB73ULL, 0x42D561B3E6243D8AULL};

struct Row {
  float top;     // the largest logit
  float ch, cl;  // log2(e) / temperature
};

// A logit as an unsigned number that falls as the logit rises; kNone for what
// is no candidate.
__device__ __forceinline__ uint32_t order_key(float l) {
  if (!(l > -INFINITY)) return kNone;
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 is 0
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k : ~k & 0x7FFFFFFFu);
}

// Where a candidate that is not the largest lies: its bin, that of y rounded to
// binary32 (which no order of two logits changes), and its weight in it, 2^(bin
// / 16) w = 1 - z', as g = z' + 2^-16 in units of 2^-33: z' is -2^-16.9 to 0.0425. (y
// is up to 3 2^-18 off its first number: half a step of the product, of the
// difference and of log2(e) / temperature, each 2^-24 of y < 64 at most.)
// Far is y from the last bin's beginning on (the far bin): such weights together are
// below 2^-42 of the largest's. Straight code, whose results then mean nothing.
constexpr int kFar = kBins - 1;
constexpr float kFarY = kFar / 16.0f;  // as in_bins() has it
constexpr int kIndexDigits = 10;  // 2^20 indices in kBins
constexpr uint32_t kShift = 1u << 17;
// y in two numbers, of which the first is negative here, of two logits: the
// difference in two numbers, times log2(e) / temperature in two.
__device__ __forceinline__ void distance2(const Row& r, F2 l, F2& yh, F2& yl) {
  const F2 top = pack2(r.top, r.top), ch = pack2(r.ch, r.ch), cl = pack2(r.cl, r.cl);
  const F2 minus = pack2(-1.0f, -1.0f);
  const F2 s = fma2(l, minus, top), bb = fma2(s, minus, top);
  const F2 e = add2(fma2(add2(s, bb), minus, top), fma2(l, minus, bb));
  yh = mul2(s, pack2(-r.ch, -r.ch));
  yl = fma2(e, ch, fma2(s, cl, fma2(s, ch, yh)));
}
// The bin and the weight of minus y = yh - yl.
__device__ __forceinline__ void split(float yh, float yl, int& bin, uint32_t& g) {
  // y = bin / 16 + x, x in units of 2^-34, from its two parts; adding 2^23
  // rounded down is a floor, adding 3 2^22 a rounding (of 3 2^16 at most)
  const float t = __fmaf_rd(yh, -16.0f, 0x1p23f);
  bin = (int)(__float_as_uint(t) & 0x7FFFFFu);
  const float xh = fmaf(t - 0x1p23f, -0.0625f, -yh);
  const int x = __float2int_rn(xh * 0x1p34f) +
                (__float_as_int(fmaf(yl, 0x1p34f, 0x1.8p23f)) - 0x4B400000);
  // 1 - 2^-x = 1 - exp(-z) = z - z^2 (1/2 - z (1/6 - z (1/24 - z / 120))), z = x
  // ln 2; z^6 / 720 < 2^-36 is left out. What follows z is below 2^-10, and
  // binary32 holds it to 2^-34.
  const int z = __mulhi(x, 0x58B90BFC);  // units of 2^-33
  const float zf = (float)z, f = zf * -0x1p-33f;
  const float q =
      fmaf(f, fmaf(f, fmaf(f, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f), 0.5f);
  const float tail = fmaf(-f * zf, q, 0x1p23f);
  g = (uint32_t)z - __float_as_uint(tail) + (0x4B000000u + kShift);
}
__device__ __forceinline__ int place(const Row& r, float l, uint32_t& g) {
  F2 h, w;
  distance2(r, pack2(l, l), h, w);
  float yh, yl, same;
  unpack2(h, yh, same);
  unpack2(w, yl, same);
  if (l == r.top || !(yh > -kFarY)) {
    g = kShift;
    return l == r.top ? 0 : kFar;
  }
  int bin;
  split(yh, yl, bin, g);
  return bin;
}
// The weights of n tokens of a bin whose g sum up to g, in units of 2^-33.
__device__ __forceinline__ uint64_t weights(uint64_t n, uint64_t g) {
  return (n << 33) + n * kShift - g;
}

// A sum of weights within a bin (1 is 2^33) in units of 2^-42 of the largest.
__device__ __forceinline__ uint64_t mass_of(int bin, uint64_t sum) {
  const uint64_t v = __umul64hi(sum << 10, kRoots[bin & 15]);
  const int n = bin >> 4;
  return n == 0 ? v : (v + ((uint64_t)1 << (n - 1))) >> n;
}

// Whether such a sum is at least `least`, in units of 2^-62 of the largest.
__device__ __forceinline__ bool at_least(int bin, uint64_t sum, uint64_t least) {
  return __umul64hi(sum << 30, kRoots[bin & 15]) >> (bin >> 4) >= least;
}

// y in bins.
__device__ __forceinline__ float in_bins(const Row& r, float l) {
  return (r.top - l) * (r.ch * 16.0f);
}
// Whether a logit's bin is this one (not the far one).
__device__ __forceinline__ bool in_bin(const Row& r, float l, int bin) {
  const float v = in_bins(r, l);
  return (v >= (float)bin && v < (float)(bin + 1)) || (bin == 0 && l == r.top);
}

// A row's settings, as the kernel works with them. (GB300 has few binary64
// units: a division by all of a block takes microseconds. What binary64 is
// needed for is done by the host, by one warp, or in pairs of binary32.)
struct Settings {
  float ch, cl;    // log2(e) / temperature, in two numbers
  bool cold;       // the first token, whatever u
  uint64_t top_k;  // 0: no limit
  double top_p;    // 1: no limit
  uint64_t min_w;  // the least weight that is kept, in units of 2^-62; 0: no limit
};
constexpr double kLog2eD = 1.4426950408889634;
constexpr float kLog2eHi = (float)kLog2eD, kLog2eLo = (float)(kLog2eD - (double)kLog2eHi);

template <class T>
struct SampleIn {
  int64_t vocab;
  const T* logits;
  int64_t stride;
  const float* u;
  Settings all;  // for every row, but for what has an array
  const float *temperatures, *top_ps, *min_ps;
  const void* top_ks;
  int32_t index_bytes;

  __device__ __forceinline__ Settings of(int64_t row) const {
    Settings s = all;
    if (temperatures != nullptr) {
      const float t = temperatures[row];
      s.cold = !(t > 0.0f);
      s.ch = fminf(kLog2eHi / t, 1e37f);
      s.cl = (fmaf(-s.ch, t, kLog2eHi) + kLog2eLo) / t;
      if (!(fabsf(s.cl) < s.ch)) s.cl = 0.0f;  // the ends of the range
    }
    if (top_ks != nullptr) {
      const int64_t k = load_index(top_ks, index_bytes, row);
      s.top_k = k > 0 ? (uint64_t)k : 0;
    }
    if (top_ps != nullptr) {
      const float p = top_ps[row];
      s.top_p = p < 1.0f ? (double)fmaxf(p, 0.0f) : 1.0;
    }
    if (min_ps != nullptr) {
      const float p = min_ps[row];
      s.min_w = p > 0.0f ? __float2ull_ru(fminf(p, 1.0f) * 0x1p62f) : 0;
    }
    return s;
  }
  __device__ __forceinline__ uint64_t uniform(int64_t row) const {  // in units of 2^-64
    const float v = u[row];
    return v > 0.0f ? __float2ull_rn(fminf(v, 1.0f - 0x1p-24f) * 0x1p64f) : 0;
  }
};

// What the leader tells the others.
struct Message {
  int bin;          // the bin that is looked into
  uint32_t lo, hi;  // and the keys
  uint32_t number;  // of tokens there
};

struct Shared {
  union {
    struct {
      uint32_t cnt[kBins], sum[kBins];  // this slice's histogram, of add()
    };
    struct {
      uint32_t kept[kBins];  // (a histogram of numbers is still read when the list is begun)
      uint64_t list[kList], sums[kList];  // leader: gathered tokens, and their running sums
      uint16_t bin_of[kList];
      uint16_t first_in[kBins];  // where a bin's tokens begin
    };
  };
  uint64_t mass[kBins + 1];     // the sums before a bin
  uint32_t before[kBins + 1];   // the tokens before it
  uint32_t chosen[kBins / 32];  // bins whose tokens are gathered
  uint32_t number, from, to;    // of those tokens and bins
  uint32_t listed;
  uint64_t warp[2][kThreads / 32];
  uint64_t said[2][kMostBlocks];  // by block
  uint64_t part[2];               // leader
  uint64_t want;                  // leader: what a border is looked for
  int limit_bin, floor_bin;       // of top_k and the first of min_p, kBins without one
  Message message[2];             // one is read while the other is written
  int found;
};

extern __shared__ __align__(16) char sample_shared[];
constexpr size_t kFixed = (sizeof(Shared) + 15) / 16 * 16;
// (By its own name: through a pointer that a function is handed, the compiler
// would not know the memory, and its atomics took five times as long.)
#define sh (*reinterpret_cast<Shared*>(sample_shared))

template <class T>
struct Sampler {
  static constexpr int E = 16 / sizeof(T);  // elements of an access to memory
  const SampleIn<T>& in;
  const int rank, blocks;
  const T* x;        // this slice
  bool held;         // whether shared memory has a copy
  int n;             // its length
  int start;         // its first index
  bool wide;         // on 16 bytes
  Row r;
  mutable int turn = 0;  // of the messages

  __device__ Sampler(const SampleIn<T>& i, int rk, int bl) : in(i), rank(rk), blocks(bl) {}
  static __device__ __forceinline__ T* copy() {
    return reinterpret_cast<T*>(sample_shared + kFixed);
  }

  __device__ __forceinline__ void sync() const {
    if (blocks > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  // All of the cluster's blocks have begun, once this has been waited for.
  __device__ __forceinline__ void begin() const {
    if (blocks > 1) cluster_arrive();
  }
  __device__ __forceinline__ void begun() const {
    if (blocks > 1) cluster_wait();
  }
  template <class V>
  __device__ __forceinline__ V* at(V* p, int block) const {
    return blocks > 1 ? cg::this_cluster().map_shared_rank(p, block) : p;
  }

  // f(logits, index of the first) of every element of the slice, kBatch at a
  // time; NaN stands for what is behind the end. (Straight code on several
  // elements side by side hides its latencies: with one after the other, a
  // block's sixteen warps issued one instruction a clock.)
  static constexpr int kBatch = 4;
  struct Batch {
    uint32_t w[kBatch * sizeof(T) / 4];
    __device__ __forceinline__ void unpack(float (&v)[kBatch]) const {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) v[k] = element(w, k);
    }
  };
  using Words = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
  static __device__ __forceinline__ float element(const uint32_t* w, int k) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(k % 2 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    else
      return __half2float(__ushort_as_half((unsigned short)(w[k / 2] >> (k % 2 * 16))));
  }
  // Elements i to i + kBatch of p, aligned on their bytes.
  static __device__ __forceinline__ Batch aligned(const T* p, int i) {
    return __builtin_bit_cast(Batch, *reinterpret_cast<const Words*>(p + i));
  }
  // The same of any p, NaN from `end` on.
  static __device__ __forceinline__ Batch guarded(const T* p, int i, int end, bool wide) {
    if (wide && i + kBatch <= end) return aligned(p, i);
    T v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) v[k] = i + k < end ? p[i + k] : from_f32<T>(NAN);
    Batch b;
    memcpy(&b, v, sizeof(b));
    return b;
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    const T* const from = x;  // (copies: what f writes might be these, for the compiler)
    const int end = n, first = start;
    const bool on16 = wide;
    constexpr int step = kBatch * kThreads;
    float l[kBatch];
    if (held) {
#pragma unroll 1
      for (int i = threadIdx.x * kBatch; i < end; i += step) {
        aligned(copy(), i).unpack(l);
        f(l, first + i);
      }
    } else {  // the next ones are read while f works on these
      Batch next = guarded(from, threadIdx.x * kBatch, end, on16);
#pragma unroll 1
      for (int i = threadIdx.x * kBatch; i < end; i += step) {
        next.unpack(l);
        next = guarded(from, i + step, end, on16);
        f(l, first + i);
      }
    }
  }

  // The slice into shared memory; gives the thread's largest element.
  __device__ __forceinline__ float load() const {
    float top = -INFINITY;
    const int whole = wide ? n / E * E : 0;
#pragma unroll 4
    for (int i = threadIdx.x * E; i < whole; i += kThreads * E) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(x + i));
      if (held) *reinterpret_cast<uint4*>(copy() + i) = q;
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < E; ++k) top = fmaxf(top, element(w, k));
    }
#pragma unroll 4
    for (int i = whole + threadIdx.x; i < n; i += kThreads) {
      const T v = x[i];
      if (held) copy()[i] = v;
      top = fmaxf(top, to_f32(v));
    }
    if (held && threadIdx.x < kBatch && n + threadIdx.x < (n + kBatch - 1) / kBatch * kBatch)
      copy()[n + threadIdx.x] = from_f32<T>(NAN);
    return top;
  }

  // ------------------------------------------------ sums and extremes
  // (Extremes are of values whose order is that of unsigned numbers.)
  template <bool kMin>
  __device__ uint64_t extreme(uint64_t v, int slot) const {  // over the cluster
#pragma unroll
    for (int s = 16; s > 0; s /= 2) {
      const uint64_t o = __shfl_xor_sync(~0u, v, s);
      v = kMin ? min(v, o) : max(v, o);
    }
    if (threadIdx.x % 32 == 0) sh.warp[slot][threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
      v = sh.warp[slot][threadIdx.x % (kThreads / 32)];
#pragma unroll
      for (int s = 16; s > 0; s /= 2) {
        const uint64_t o = __shfl_xor_sync(~0u, v, s);
        v = kMin ? min(v, o) : max(v, o);
      }
      if (threadIdx.x < blocks) *at(&sh.said[slot][rank], threadIdx.x) = v;
    }
    sync();
    v = sh.said[slot][0];
    for (int b = 1; b < blocks; ++b) v = kMin ? min(v, sh.said[slot][b]) : max(v, sh.said[slot][b]);
    return v;
  }

  // What a histogram's bins are.
  enum Digit {
    kCount,  // those of place(), and only the number of tokens
    kPlace,  // those of place(), their sums as masses
    kKey,    // the keys lo..hi of m.bin, from lo on, 2^shift a bin
    kIndex,  // the indices with the key lo, 1024 a bin
  };
  // Leaves the running sums (in a bin's own units, but for kPlace). clean: the
  // bins are empty.
  __device__ __forceinline__ void clear() const {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.cnt[i] = sh.sum[i] = 0;
  }
  __device__ __noinline__ void histogram(Digit digit, const Message& m, int shift,
                                         bool clean = false) const {
    if (!clean) {
      __syncthreads();  // what the leader reads of its list is read
      clear();
    }
    __syncthreads();
    uint32_t tops = 0, fars = 0;
    const Row row = r;
    // A bin's sum of g, below 2^46 in a slice, has its low 32 bits in sum; cnt
    // counts its overflows above the number of tokens. (Two additions an element:
    // with three 64 rows of 262,144 took 106 us for 102, with one of 64 bits 150.)
    const auto add = [](int d, uint32_t g, uint32_t n) {
      const uint32_t old = atomicAdd(&sh.sum[d], g);
      atomicAdd(&sh.cnt[d], n + (old + g < old ? kOverflow : 0));
    };
    if (digit == kCount) {
      each([&, row](const float (&l)[kBatch], int) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float v = in_bins(row, l[k]);
          const bool close = v < (float)kFar, top = l[k] == row.top;
          tops += top;
          fars += !close && !top && l[k] > -INFINITY;
          if (close && !top) atomicAdd(&sh.cnt[(int)v], 1u);
        }
      });
    } else if (digit == kPlace) {
      each([&, row](const float (&l)[kBatch], int) {
        uint32_t g[kBatch];
        int d[kBatch];
        float yh[kBatch], yl[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; k += 2) {
          F2 h, w;
          distance2(row, pack2(l[k], l[k + 1]), h, w);
          unpack2(h, yh[k], yh[k + 1]);
          unpack2(w, yl[k], yl[k + 1]);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) split(yh[k], yl[k], d[k], g[k]);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (yh[k] > -kFarY && l[k] != row.top) add(d[k], g[k], 1);
          else if (l[k] == row.top) ++tops;  // many may be alike there
          else fars += l[k] > -INFINITY;
        }
      });
    } else {
      const int bin = m.bin;
      const uint32_t lo = m.lo, hi = m.hi;
      each([&, row](const float (&l)[kBatch], int i) {
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k, ++i) {
          if (!in_bin(row, l[k], bin)) continue;
          const uint32_t key = order_key(l[k]);
          if (key < lo || key > hi) continue;
          uint32_t g;
          place(row, l[k], g);
          add(digit == kKey ? (int)((key - lo) >> shift) : i >> kIndexDigits, g, 1);
        }
      });
    }
    fars = __reduce_add_sync(~0u, fars);
    tops = __reduce_add_sync(~0u, tops);
    if (threadIdx.x % 32 == 0) {
      if (tops) add(0, tops * kShift, tops);
      if (fars) atomicAdd(&sh.cnt[kFar], fars);
    }
    sync();
    if (digit == kCount) {  // every block adds up all of them
      for (int i = threadIdx.x; i < kBins; i += kThreads) {
        uint32_t c[kMostBlocks], n = 0;
#pragma unroll
        for (int b = 0; b < kMostBlocks; ++b) c[b] = b < blocks ? at(sh.cnt, b)[i] : 0;
#pragma unroll
        for (int b = 0; b < kMostBlocks; ++b) n += c[b];
        sh.before[i] = n;
        sh.mass[i] = 0;
      }
      __syncthreads();
      running_sums();
      return;
    }
    // each block adds up a part of the bins, and tells the others
    const int share = kBins / blocks;
    for (int i = rank * share + threadIdx.x; i < (rank + 1) * share; i += kThreads) {
      uint32_t c[kMostBlocks], lo[kMostBlocks], n = 0;
      uint64_t g = 0;
#pragma unroll
      for (int b = 0; b < kMostBlocks; ++b) {
        c[b] = b < blocks ? at(sh.cnt, b)[i] : 0;
        lo[b] = b < blocks ? at(sh.sum, b)[i] : 0;
      }
#pragma unroll
      for (int b = 0; b < kMostBlocks; ++b) {
        n += c[b] % kOverflow;
        g += ((uint64_t)(c[b] / kOverflow) << 32) + lo[b];
      }
      uint64_t w = weights(n, g);
      if (digit == kPlace) w = i == kFar ? 0 : mass_of(i, w);
      for (int b = 0; b < blocks; ++b) {
        at(sh.before, b)[i] = n;
        at(sh.mass, b)[i] = w;
      }
    }
    sync();
    running_sums();
  }

  // before and mass: from what a bin holds to what is before it
  __device__ void running_sums() const {
    constexpr int per = kBins / kThreads;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uint32_t c[per], ct = 0;
    uint64_t m[per], mt = 0;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      c[k] = sh.before[tid * per + k];
      m[k] = sh.mass[tid * per + k];
      ct += c[k];
      mt += m[k];
    }
    uint32_t ci = ct;
    uint64_t mi = mt;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const uint32_t a = __shfl_up_sync(~0u, ci, s);
      const uint64_t b = __shfl_up_sync(~0u, mi, s);
      if (lane >= s) ci += a, mi += b;
    }
    if (lane == 31) sh.warp[0][warp] = ci, sh.warp[1][warp] = mi;
    __syncthreads();
    uint32_t cb = ci - ct;
    uint64_t mb = mi - mt;
    for (int w = 0; w < warp; ++w) cb += (uint32_t)sh.warp[0][w], mb += sh.warp[1][w];
#pragma unroll
    for (int k = 0; k < per; ++k) {
      sh.before[tid * per + k] = cb;
      sh.mass[tid * per + k] = mb;
      cb += c[k];
      mb += m[k];
    }
    if (tid == kThreads - 1) sh.before[kBins] = cb, sh.mass[kBins] = mb;
    __syncthreads();
  }

  // Leader: the first bin up to which holds(number, sum) is true. before() is
  // run by one thread first (GB300 has few binary64 units: a rounding of
  // top_p times a sum by all of a block takes microseconds).
  template <class F>
  __device__ int first_bin(F holds) const {
    return first_bin([] {}, holds);
  }
  template <class G, class F>
  __device__ int first_bin(G before, F holds) const {
    __syncthreads();
    if (threadIdx.x == 0) {
      before();
      sh.found = kBins - 1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads)
      if (holds(sh.before[i + 1], sh.mass[i + 1]) && (i == 0 || !holds(sh.before[i], sh.mass[i])))
        sh.found = i;
    __syncthreads();
    return sh.found;
  }

  // The leader's message, to all.
  __device__ __forceinline__ void tell(const Message& m) const {
    if (threadIdx.x < blocks) *at(&sh.message[turn], threadIdx.x) = m;
    if (threadIdx.x == 0) sh.listed = 0;  // of the gather that may follow
  }
  __device__ __forceinline__ Message hear() const {
    sync();
    const Message m = sh.message[turn];
    turn ^= 1;
    return m;
  }

  // Leader: the list sorted, with the running sums of its weights, in a bin's
  // units or (masses) all in one; `number` of it.
  __device__ __noinline__ void sort(int number, bool masses) const {
    if (number <= kRanked) {  // each finds its rank among all
      uint64_t mine = 0;
      int place_ = 0;
      const bool one = threadIdx.x < number;
      if (one) {
        mine = sh.list[threadIdx.x];
#pragma unroll 8
        for (int i = 0; i < number; ++i) place_ += sh.list[i] < mine;
      }
      __syncthreads();
      if (one) sh.list[place_] = mine;
    }
    int size = 2;
    while (size < number) size *= 2;
    if (number <= kRanked) size = 0;
    for (int i = number + threadIdx.x; i < size; i += kThreads) sh.list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2) {
      for (int j = k / 2; j > 0; j /= 2) {
        for (int p = threadIdx.x; p < size / 2; p += kThreads) {
          const int i = 2 * p - (p & (j - 1)), o = i + j;
          const uint64_t a = sh.list[i], b = sh.list[o];
          if ((a > b) == ((i & k) == 0)) sh.list[i] = b, sh.list[o] = a;
        }
        __syncthreads();
      }
    }
    constexpr int per = kList / kThreads;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uint64_t m[per], mt = 0;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      const int i = tid * per + k;
      m[k] = 0;
      if (i < number) {
        uint32_t g;
        const int bin = place(r, key_logit((uint32_t)(sh.list[i] >> 32)), g);
        m[k] = weights(1, g);
        if (masses) {
          m[k] = bin == kFar ? 0 : mass_of(bin, m[k]);
          sh.bin_of[i] = (uint16_t)bin;
        }
      }
      mt += m[k];
    }
    uint64_t mi = mt;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const uint64_t b = __shfl_up_sync(~0u, mi, s);
      if (lane >= s) mi += b;
    }
    if (lane == 31) sh.warp[0][warp] = mi;
    __syncthreads();
    uint64_t mb = mi - mt;
    for (int w = 0; w < warp; ++w) mb += sh.warp[0][w];
#pragma unroll
    for (int k = 0; k < per; ++k) {
      mb += m[k];
      if (tid * per + k < number) sh.sums[tid * per + k] = mb;  // the element's own included
    }
    __syncthreads();
  }
  __device__ __forceinline__ uint64_t weight_in_bin(uint32_t key) const {
    uint32_t g;
    place(r, key_logit(key), g);
    return weights(1, g);
  }

  // What a border is the first place of: n tokens, or a mass of `want` with
  // `base` before the bin.
  struct Goal {
    bool count;
    int bin;
    uint64_t want, base;
    __device__ __forceinline__ bool operator()(uint64_t n, uint64_t sum) const {
      return count ? n >= want : base + mass_of(bin, sum) >= want;
    }
  };
  // A border in a bin.
  struct Border {
    int bin;
    uint64_t number;  // tokens of the bin up to it
    uint64_t sum;     // their weights
    int64_t token;    // the last of them, where it was asked for
  };

  // The place in `bin` (of `number` tokens) that is the first where
  // holds(number, sum) of the bin's tokens up to it. bin, number (0: nothing to
  // be done) and holds are the leader's, as is the result; all blocks call it.
  // used: whether the leader's running sums are gone.
  __device__ __noinline__ Border look(int bin, uint32_t number, bool pick, bool& used,
                                      Goal holds) const {
    Border out = {bin, 0, 0, -1};
    uint64_t nb = 0, sb = 0;  // tokens and weights before the keys lo..hi
    uint32_t lo = 0, hi = kNone - 1;
    if (rank == 0) tell({bin, lo, hi, number});
    Message m = hear();
    if (m.number == 0) return out;
    used = used || m.number > kList;
    while (m.number > kList) {
      uint64_t kmin = kNone, kmax = 0;
      each([&](const float (&l)[kBatch], int) {
#pragma unroll 1
        for (int j = 0; j < kBatch; ++j) {
          if (!in_bin(r, l[j], m.bin)) continue;
          const uint32_t k = order_key(l[j]);
          if (k < m.lo || k > m.hi) continue;
          kmin = min(kmin, (uint64_t)k);
          kmax = max(kmax, (uint64_t)k);
        }
      });
      m.lo = (uint32_t)extreme<true>(kmin, 0);
      m.hi = (uint32_t)extreme<false>(kmax, 1);
      if (m.lo == m.hi) return alike(m, nb, sb, pick, holds);
      int shift = 32 - __clz(m.hi - m.lo) - 10;
      if (shift < 0) shift = 0;
      histogram(kKey, m, shift);
      if (rank == 0) {
        const int d = first_bin([&](uint32_t c, uint64_t s) { return holds(nb + c, sb + s); });
        const uint32_t many = sh.before[d + 1] - sh.before[d];
        nb += sh.before[d];
        sb += sh.mass[d];
        lo = m.lo + ((uint32_t)d << shift);
        hi = min(m.hi, lo + ((uint32_t)1 << shift) - 1);  // (keys past m.hi are not counted)
        tell({bin, lo, hi, many});
      }
      m = hear();
    }
    gather(m, false);
    if (rank == 0) {
      sort((int)m.number, false);
      if (threadIdx.x == 0) sh.found = (int)m.number - 1;
      __syncthreads();
      for (int i = threadIdx.x; i < (int)m.number; i += kThreads)
        if (holds(nb + i + 1, sb + sh.sums[i]) && (i == 0 || !holds(nb + i, sb + sh.sums[i - 1])))
          sh.found = i;
      __syncthreads();
      out.number = nb + sh.found + 1;
      out.sum = sb + sh.sums[sh.found];
      out.token = (int64_t)(uint32_t)sh.list[sh.found];
    }
    return out;
  }

  // Collects the tokens of m.bin with keys lo..hi in the leader's list; of one
  // key: those whose index is in [1024 bin, 1024 (bin + 1)).
  __device__ __noinline__ void gather(const Message& m, bool one) const {
    uint32_t* listed = at(&sh.listed, 0);
    uint64_t* list = at(sh.list, 0);
    const Row row = r;
    const int bin = m.bin;
    const uint32_t lo = m.lo, hi = m.hi;
    each([=](const float (&l)[kBatch], int i) {
#pragma unroll 1
      for (int j = 0; j < kBatch; ++j, ++i) {
        if (one ? i >> kIndexDigits != bin : !in_bin(row, l[j], bin)) continue;
        const uint32_t k = order_key(l[j]);
        if (k < lo || k > hi) continue;
        const uint32_t to = atomicAdd(listed, 1u);
        if (to < (uint32_t)kList) list[to] = (uint64_t)k << 32 | (uint32_t)i;
      }
    });
    sync();
  }
  // The same for all tokens of bins up to `to` (few), or of the chosen ones, which
  // are of bins from..to.
  __device__ __noinline__ void gather_chosen(bool few, int from, int to) const {
    uint32_t* listed = at(&sh.listed, 0);
    uint64_t* list = at(sh.list, 0);
    const Row row = r;
    const auto add = [=](float l, int i) {
      const uint32_t at = atomicAdd(listed, 1u);
      if (at < (uint32_t)kList) list[at] = (uint64_t)order_key(l) << 32 | (uint32_t)i;
    };
    if (few) {
      const float limit = (float)(to + 1);
      each([=](const float (&l)[kBatch], int i) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (in_bins(row, l[k]) < limit || l[k] == row.top) add(l[k], i + k);
      });
    } else {
      const float low = (float)from, high = (float)(to + 1);
      const bool tops = from == 0;
      each([=](const float (&l)[kBatch], int i) {
        bool may[kBatch];
        bool any = false;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float v = in_bins(row, l[k]);
          may[k] = (v >= low && v < high) || (tops && l[k] == row.top);
          any = any || may[k];
        }
        if (!any) return;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int b = l[k] == row.top ? 0 : (int)in_bins(row, l[k]);
          if (may[k] && (sh.chosen[b / 32] >> b % 32 & 1)) add(l[k], i + k);
        }
      });
    }
    sync();
  }

  // A warp: the first of n for which holds(i) (and for all after it), or n.
  template <class F>
  __device__ __forceinline__ int first_of(int n, F holds) const {
    int lo = 0, hi = n;
    const int lane = threadIdx.x % 32;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32, i = lo + step * (lane + 1) - 1;
      const uint32_t yes = __ballot_sync(~0u, i >= hi || holds(i));
      if (yes == 0) return hi;
      const int k = __ffs(yes) - 1;
      hi = min(hi, lo + step * (k + 1) - 1);
      lo += step * k;
    }
    return lo;
  }

  // Masses that borders are looked for: p kept, rounded up, and at least 1, as the
  // first is kept (the product is one of binary64, where 0.9 of 10 is 9); the
  // first that exceeds u kept, u in units of 2^-64.
  static __device__ __forceinline__ uint64_t share(double p, uint64_t kept) {
    return max((unsigned long long)ceil(p * (double)kept), 1ull);
  }
  static __device__ __forceinline__ uint64_t beyond(uint64_t u, uint64_t kept) {
    return __umul64hi(u, kept) + 1;
  }
  struct Limits : Settings {
    uint64_t u;
  };

  // A block's first warp: the bins in which the borders lie, as far as bins tell.
  // A border's bin hangs on the sum of what the one before it
  // keeps, of which a lower and an upper limit are known: all bins between.
  // number 0: more tokens than the list holds.
  __device__ __noinline__ void plan(const Limits& lim) const {
    const int lane = threadIdx.x % 32;
    uint32_t mine[kBins / 32 / 32] = {};  // of the chosen bins: words lane, lane + 32
    uint32_t number = 0;
    const auto choose = [&](int from, int to) {
#pragma unroll
      for (int k = 0; k < kBins / 32 / 32; ++k) {
        const int w = (k * 32 + lane) * 32;
        const int a = max(from - w, 0), b = min(to - w, 31);
        if (a <= b) mine[k] |= (~0u >> (31 - (b - a))) << a;
      }
    };
    const auto bin_of_mass = [&](uint64_t want) {
      return min(first_of(kBins, [&](int i) { return sh.mass[i + 1] >= want; }), kBins - 1);
    };
    uint64_t lo = sh.mass[kBins], hi = lo;  // of the sum that is kept
    int end = kBins, limit = kBins, floor_ = kBins;
    if (lim.top_k > 0 && lim.top_k < sh.before[kBins]) {
      const int d = first_of(kBins, [&](int i) { return sh.before[i + 1] >= lim.top_k; });
      limit = end = d;
      lo = sh.mass[d];
      hi = sh.mass[d + 1];
      if (d != kFar) choose(d, d);  // (the far bin weighs nothing)
    }
    if (lim.top_p < 1.0) {
      const int a = bin_of_mass(share(lim.top_p, lo)), b = bin_of_mass(share(lim.top_p, hi));
      choose(a, b);
      end = min(end, b);
      lo = sh.mass[a];
      hi = min(hi, sh.mass[b + 1]);
    }
    if (lim.min_w != 0) {
      // (A weight passes its bin's ends by less than 2^-16 of itself: one near an end
      // may be in the bin before or after.) The last bin that may hold weights of
      // min_w, and the first that may hold smaller ones.
      const int d = first_of(kFar, [&](int i) {
                      return !at_least(i, (1ull << 33) + kShift, lim.min_w);
                    }) - 1;
      const int c = first_of(d, [&](int i) {
        return !at_least(i + 1, (1ull << 33) - kShift, lim.min_w);
      });
      if (c <= end) {
        floor_ = c;
        choose(c, d);
        lo = min(lo, sh.mass[c]);
        hi = min(hi, sh.mass[d + 1]);
      }
    }
    choose(bin_of_mass(beyond(lim.u, lo)), bin_of_mass(beyond(lim.u, hi)));
#pragma unroll
    for (int k = 0; k < kBins / 32 / 32; ++k) {
      const int w = k * 32 + lane;
      for (uint32_t left = mine[k]; left != 0; left &= left - 1) {
        const int d = w * 32 + __ffs(left) - 1;
        number += sh.before[d + 1] - sh.before[d];
      }
      sh.chosen[w] = mine[k];
    }
    number = __reduce_add_sync(~0u, number);
    uint32_t least = kBins, most = 0;
#pragma unroll
    for (int k = 0; k < kBins / 32 / 32; ++k) {
      if (mine[k] == 0) continue;
      least = min(least, (uint32_t)((k * 32 + lane) * 32 + __ffs(mine[k]) - 1));
      most = max(most, (uint32_t)((k * 32 + lane) * 32 + 31 - __clz(mine[k])));
    }
    least = __reduce_min_sync(~0u, least);
    most = __reduce_max_sync(~0u, most);
    if (lane == 0) {
      sh.limit_bin = limit;
      sh.floor_bin = floor_;
      sh.number = number > (uint32_t)kList ? 0 : number;
      sh.from = least;
      sh.to = most;
    }
  }

  // Leader: the token, of the first m.number tokens of all.
  __device__ __noinline__ int64_t among_few(int number, const Limits& lim) const {
    sort(number, true);
    if (threadIdx.x >= 32) return -1;
    int n = (int)min((uint64_t)number, lim.top_k);
    if (lim.top_p < 1.0) {
      const uint64_t want = share(lim.top_p, sh.sums[n - 1]);
      n = min(n, 1 + first_of(n, [&](int i) { return sh.sums[i] >= want; }));
    }
    if (lim.min_w != 0)
      n = max(1, first_of(n, [&](int i) { return !heavy((uint32_t)(sh.list[i] >> 32), lim); }));
    const uint64_t want = beyond(lim.u, sh.sums[n - 1]);
    const int i = first_of(n, [&](int k) { return sh.sums[k] >= want; });
    return (int64_t)(uint32_t)sh.list[min(i, n - 1)];
  }

  // Leader: the token, where the list has all tokens of the bins of plan().
  __device__ __noinline__ int64_t among_chosen(int number, const Limits& lim) const {
    sort(number, true);
    // sums from the row's first token on; a bin's last one agrees with its sum
    for (int i = threadIdx.x; i < number; i += kThreads)
      if (i == 0 || sh.bin_of[i] != sh.bin_of[i - 1]) sh.first_in[sh.bin_of[i]] = (uint16_t)i;
    __syncthreads();
    uint64_t sum[kList / kThreads];
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i >= number) continue;
      const int d = sh.bin_of[i], f = sh.first_in[d];
      sum[k] = sh.mass[d] + sh.sums[i] - (f > 0 ? sh.sums[f - 1] : 0);
      if (i + 1 == number || sh.bin_of[i + 1] != d) sum[k] = sh.mass[d + 1];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i < number) sh.sums[i] = sum[k];
    }
    __syncthreads();
    if (threadIdx.x >= 32) return -1;
    const auto place_of = [&](int i) {  // tokens up to this one
      const int d = sh.bin_of[i];
      return sh.before[d] + (uint32_t)(i - sh.first_in[d] + 1);
    };
    const auto reaches = [&](uint64_t want) {
      return min(number - 1, first_of(number, [&](int i) { return sh.sums[i] >= want; }));
    };
    uint64_t kept = sh.mass[kBins];
    uint32_t end = sh.before[kBins];
    if (sh.limit_bin == kFar) {
      end = (uint32_t)lim.top_k;
    } else if (sh.limit_bin < kBins) {
      const int i = min(number - 1, first_of(number, [&](int k) {
                          return place_of(k) >= (uint32_t)lim.top_k;
                        }));
      end = place_of(i);
      kept = sh.sums[i];
    }
    if (lim.top_p < 1.0) {
      const int i = reaches(share(lim.top_p, kept));
      end = place_of(i);
      kept = sh.sums[i];
    }
    if (sh.floor_bin < kBins) {
      const int d = sh.floor_bin;
      const int j =
          first_of(number, [&](int i) { return !heavy((uint32_t)(sh.list[i] >> 32), lim); });
      const bool in = j > 0 && sh.bin_of[j - 1] >= d;  // else none from its bin on
      const uint32_t many = in ? place_of(j - 1) : sh.before[d];
      if (many < end) kept = in ? sh.sums[j - 1] : sh.mass[d];
    }
    return (int64_t)(uint32_t)sh.list[reaches(beyond(lim.u, kept))];
  }

  // look() among m.number tokens of one logit (the key m.lo), more than can be
  // sorted.
  __device__ __noinline__ Border alike(Message m, uint64_t nb, uint64_t sb, bool pick,
                                       Goal holds) const {
    Border out = {m.bin, 0, 0, -1};
    const uint64_t w = weight_in_bin(m.lo);
    uint32_t lo = 1, hi = m.number;  // the first for which it holds
    if (rank == 0) {
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (holds(nb + mid, sb + mid * w)) hi = mid;
        else lo = mid + 1;
      }
      out.number = nb + lo;
      out.sum = sb + lo * w;
    }
    if (!pick) return out;
    // the lo-th by index
    histogram(kIndex, m, 0);
    if (rank == 0) {
      const int d = first_bin([&](uint32_t c, uint64_t) { return c >= lo; });
      tell({d, m.lo, m.lo, sh.before[d + 1] - sh.before[d]});
      lo -= sh.before[d];
    }
    m = hear();
    gather(m, true);
    if (rank == 0) {
      sort((int)m.number, false);
      out.token = (int64_t)(uint32_t)sh.list[lo - 1];
    }
    return out;
  }

  // Whether a key's weight is at least min_w.
  __device__ __forceinline__ bool heavy(uint32_t key, const Settings& lim) const {
    const float l = key_logit(key);
    if (!(l > -INFINITY)) return false;
    uint32_t g;
    const int bin = place(r, l, g);
    return bin != kFar && at_least(bin, weights(1, g), lim.min_w);
  }
  // The last key of which that is true (weights fall as keys rise).
  __device__ uint32_t last_key(const Settings& lim) const {
    uint32_t lo = order_key(r.top), hi = kNone - 1;  // lo always is one
    const int lane = threadIdx.x % 32;
    while (lo < hi) {
      const uint32_t step = (hi - lo + 31) / 32;
      const uint64_t k = (uint64_t)lo + (uint64_t)step * (lane + 1);
      const bool in = k <= hi && heavy((uint32_t)k, lim);
      const int many = __popc(__ballot_sync(~0u, in));
      const uint64_t next = (uint64_t)lo + (uint64_t)step * (many + 1) - 1;
      lo += step * many;
      hi = (uint32_t)min((uint64_t)hi, next);
    }
    return lo;
  }

  // Leader: number and sum of the tokens of `bin` whose key is at most `last`
  // (leader's too; 0: nothing to be done).
  __device__ Border upto(int bin, uint32_t last) const {
    Border out = {bin, 0, 0, -1};
    if (rank == 0) {
      if (threadIdx.x < 2) sh.part[threadIdx.x] = 0;
      tell({bin, 0, last, 0});
    }
    const Message m = hear();
    if (m.hi == 0) return out;
    uint64_t c = 0, s = 0;
    const Row row = r;
    each([&, row](const float (&l)[kBatch], int) {
#pragma unroll 1
      for (int k = 0; k < kBatch; ++k) {
        if (!in_bin(row, l[k], m.bin) || order_key(l[k]) > m.hi) continue;
        uint32_t g;
        place(row, l[k], g);
        ++c;
        s += weights(1, g);
      }
    });
#pragma unroll
    for (int k = 16; k > 0; k /= 2) {
      c += __shfl_xor_sync(~0u, c, k);
      s += __shfl_xor_sync(~0u, s, k);
    }
    if (threadIdx.x % 32 == 0 && c != 0) {
      atomicAdd((unsigned long long*)at(&sh.part[0], 0), (unsigned long long)c);
      atomicAdd((unsigned long long*)at(&sh.part[1], 0), (unsigned long long)s);
    }
    sync();
    if (rank == 0) out.number = sh.part[0], out.sum = sh.part[1];
    return out;
  }

  __device__ int64_t run(int64_t row);
  __device__ __noinline__ int64_t one_by_one(const Limits& lim) const;
};

template <class T>
__device__ int64_t Sampler<T>::run(int64_t row) {
  begin();
  clear();
  if (threadIdx.x == 0) sh.listed = 0;
  const Limits lim = {in.of(row), in.uniform(row)};
  const float mine = load();
  begun();
  const uint32_t top = (uint32_t)extreme<true>((uint64_t)order_key(mine), 0);
  if (top == kNone) return -1;
  r.top = key_logit(top);
  if (lim.cold || lim.top_k == 1) {
    uint64_t first = ~0ull;
    each([&](const float (&l)[kBatch], int i) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (l[k] == r.top) first = min(first, (uint64_t)(i + k));
    });
    return (int64_t)extreme<true>(first, 1);
  }
  r.ch = lim.ch;
  r.cl = lim.cl;
  // A few tokens by top_k: these and no others, from a histogram of numbers.
  bool clean = true;
  if (lim.top_k > 0 && lim.top_k <= kFew) {
    histogram(kCount, {}, 0, true);
    const int d = min(first_of(kBins, [&](int i) { return sh.before[i + 1] >= lim.top_k; }),
                      kBins - 1);
    const uint32_t n = sh.before[d + 1];
    if (n <= (uint32_t)kList && d != kFar) {
      gather_chosen(true, 0, d);
      return rank == 0 ? among_few((int)n, lim) : -1;
    }
    sync();  // others may still add up the numbers
    clean = false;
  }
  // Otherwise the borders' bins, from the sums of all.
  histogram(kPlace, {}, 0, clean);
  if (threadIdx.x < 32) plan(lim);
  __syncthreads();
  if (sh.number != 0) {
    gather_chosen(false, (int)sh.from, (int)sh.to);
    return rank == 0 ? among_chosen((int)sh.number, lim) : -1;
  }
  return one_by_one(lim);
}

// The borders one after the other, where their bins hold more tokens than the
// list: each bin is cut until its border's part fits.
template <class T>
__device__ __noinline__ int64_t Sampler<T>::one_by_one(const Limits& lim) const {
  const uint64_t top_k = lim.top_k;
  const auto bins = [&] { histogram(kPlace, {}, 0); };

  // The last bin of what is kept, how many of its tokens, and the sum of all of
  // it (the leader's; all blocks know which limits there are).
  bool used = false;
  int end = kBins;
  uint64_t number = 0, kept = rank == 0 ? sh.mass[kBins] : 0, base = 0;
  if (top_k > 0) {
    int d = 0;
    uint32_t many = 0;
    uint64_t want = 0;
    if (rank == 0 && top_k < sh.before[kBins]) {
      d = first_bin([&](uint32_t n, uint64_t) { return n >= top_k; });
      want = top_k - sh.before[d];
      many = sh.before[d + 1] - sh.before[d];
      base = sh.mass[d];
      end = d;
      number = want;
      kept = sh.mass[d + 1];
      if (d == kFar || want == many) many = 0;  // weightless, or the whole bin
    }
    const Border b = look(d, many, false, used, {true, d, want, 0});
    if (many != 0) kept = base + mass_of(d, b.sum);
  }
  if (lim.top_p < 1.0) {
    if (used) bins();
    used = false;
    int d = 0;
    uint32_t many = 0;
    uint64_t want = 0;
    if (rank == 0) {
      d = first_bin(
          [&] { sh.want = share(lim.top_p, kept); },
          [&](uint32_t, uint64_t s) { return s >= sh.want; });
      want = sh.want;
      many = sh.before[d + 1] - sh.before[d];
      base = sh.mass[d];
      end = d;
      number = many;
      kept = sh.mass[d + 1];
      if (many == 1) many = 0;
    }
    const Border b = look(d, many, false, used, {false, d, want, base});
    if (many != 0) number = b.number, kept = base + mass_of(d, b.sum);
  }
  if (lim.min_w != 0) {
    if (used) bins();
    used = false;
    int d = 0;
    uint32_t last = 0;
    if (rank == 0) {
      last = last_key(lim);
      uint32_t g;
      d = place(r, key_logit(last), g);
      base = sh.mass[d];
      if (d > end) last = 0;
    }
    const Border b = upto(d, last);
    if (last != 0 && (d < end || b.number < number)) kept = base + mass_of(d, b.sum);
  }
  if (used) bins();
  int d = 0;
  uint32_t many = 0;
  uint64_t want = 0;
  if (rank == 0) {
    d = first_bin(
        [&] { sh.want = beyond(lim.u, kept); },
        [&](uint32_t, uint64_t s) { return s >= sh.want; });
    want = sh.want;
    many = sh.before[d + 1] - sh.before[d];
    base = sh.mass[d];
  }
  return look(d, many, true, used, {false, d, want, base}).token;
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(SampleIn<T> in, int64_t* __restrict__ tokens, int blocks, int slice, bool hold,
              bool wide) {
  const int rank = (int)(blockIdx.x % (unsigned)blocks);
  const int64_t row = blockIdx.x / (unsigned)blocks;
  Sampler<T> s(in, rank, blocks);
  s.start = rank * slice;
  s.n = max(0, min(slice, (int)in.vocab - s.start));
  s.x = in.logits + row * in.stride + (s.n > 0 ? s.start : 0);
  s.held = hold;
  s.wide = wide;
  // (What a block reads or writes of another is followed by a wait for all of
  // them, so that none is gone too early.)
  const int64_t token = s.run(row);
  if (rank == 0 && threadIdx.x == 0) tokens[row] = token;
}

// Blocks a row: up to one an SM where a slice then keeps 2048 tokens, up to two
// where it keeps 8192, up to 512 blocks, of which the last wait for others to end,
// where it keeps 32,768. (Each step of a row costs a wait for all of its blocks,
// and two blocks of an SM are in each other's way.) At least so many that a
// slice's histogram stays within its 32 bits. Measured, us for blocks 1 / 2 / 4 / 8:
// of 65,536 tokens 1 row 55 / 39 / 31 / 24, 48 rows 56 / 41 / 39 / 50, 76 rows 57 /
// 44 / 57 / 70, 128 rows 60 / 58 / 74 / 100, 256 rows 90 / 107 / 131 / 189; of 10,007
// 36 rows 21 / 21 / 19 / 23, 100 rows 21 / 25 / 38 / 57; of 262,144 16 rows - / 130 /
// 62 / 72, 100 rows - / 195 / 174 / 170, 200 rows - / 281 / 265 / 320.
int sample_blocks(int64_t rows, int64_t vocab) {
  const auto worth = [&](int64_t c) {
    return rows * c <= 152 ? vocab >= c * 2048
                           : (rows * c <= 304 && vocab >= c * 8192) ||
                                 (rows * c <= 512 && vocab >= c * 32768);
  };
  int c = 1;
  while (c < kMostBlocks && (worth(2 * c) || vocab > (int64_t)c * kMostSlice)) c *= 2;
  return c;
}

}  // namespace
}  // namespace cr

extern "C" {

cr_status cr_sample(const cr_sample_args* a, int64_t* tokens, void* stream) {
  using namespace cr;
  if (a == nullptr) return CR_ERR_INVALID_ARG;
  const size_t es = model_esize(a->dt);
  if (es == 0 || a->rows < 0 || a->vocab < 0 || a->row_stride < 0 ||
      (a->top_ks != nullptr && !index_width_ok(a->index_bytes)))
    return CR_ERR_INVALID_ARG;
  if (a->rows == 0) return CR_OK;
  if (a->u == nullptr || tokens == nullptr || (a->vocab > 0 && a->logits == nullptr))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(a->logits, es) || !ptr_aligned(a->u, 4) || !ptr_aligned(tokens, 8) ||
      !ptr_aligned(a->temperatures, 4) || !ptr_aligned(a->top_ps, 4) ||
      !ptr_aligned(a->min_ps, 4) ||
      (a->top_ks != nullptr && !ptr_aligned(a->top_ks, a->index_bytes)) ||
      overwrites({tokens}, {a->logits, a->u, a->temperatures, a->top_ps, a->min_ps, a->top_ks}))
    return CR_ERR_INVALID_ARG;
  if (a->vocab > (int64_t)1 << 20 || a->rows > kMaxBlocks / kMostBlocks) return CR_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int blocks = sample_blocks(a->rows, a->vocab);
  const int slice = (int)ceil_div(ceil_div(a->vocab, blocks), 8) * 8;
  // in shared memory where two blocks an SM fit (200 rows of 65,536 in two blocks
  // each: 108 us with one, 94 with two that read their slices again from L2)
  const bool hold = kFixed + slice * es <= 112 * 1024;
  const size_t smem = kFixed + (hold ? slice * es : 0);
  const bool wide = rows_aligned(a->logits, a->row_stride, 0, es, 16);
  Settings all;
  const double c = a->temperature > 0.0 ? std::min(kLog2eD / a->temperature, 1e37) : 0.0;
  all.cold = !(a->temperature > 0.0);
  all.ch = (float)c;
  all.cl = (float)(c - (double)all.ch);
  all.top_k = a->top_k > 0 ? (uint64_t)a->top_k : 0;
  all.top_p = a->top_p < 1.0 ? std::max(a->top_p, 0.0) : 1.0;
  all.min_w = 0;
  if (a->min_p > 0.0) all.min_w = (uint64_t)std::ceil(std::ldexp(std::min(a->min_p, 1.0), 62));
  bool done = false;
  CR_MODEL_TYPE(a->dt, {
    const SampleIn<T> in = {a->vocab,  static_cast<const T*>(a->logits), a->row_stride, a->u,
                            all,       a->temperatures, a->top_ps, a->min_ps, a->top_ks,
                            a->index_bytes};
    CR_LAUNCH(kKSample, s,
              done = launch_clusters(sample_kernel<T>, a->rows * blocks, blocks, kThreads, smem, s,
                                     in, tokens, blocks, slice, hold, wide));
  });
  return done && cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
