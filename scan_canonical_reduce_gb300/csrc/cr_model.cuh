// Shared pieces of the model operators (embedding, causal convolution,
// selective scan): element types, vector access, the two nonlinearities, and
// the host-side argument checks.
//
// Tensors of 16-bit types are read and written as such; everything between
// is binary32. Rounding to 16 bits happens once, when a result is stored.
#pragma once

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cr.h"

namespace cr {

// ------------------------------------------------------------ elements
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

template <class T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

// V consecutive elements as binary32. wide: p is aligned to the whole pack
// and all V elements exist; otherwise the first `have` are read one by one
// and the rest are zero.
template <class T, int V>
__device__ __forceinline__ void load_f32(const T* p, bool wide, int have, float (&f)[V]) {
  if (wide) {
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(q.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = i < have ? to_f32(p[i]) : 0.0f;
  }
}

template <class T, int V>
__device__ __forceinline__ void store_f32(T* p, bool wide, int have, const float (&f)[V]) {
  if (wide) {
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < have) p[i] = from_f32<T>(f[i]);
  }
}

// V elements as they stand in memory, not waited for before they are used.
// kWide: consecutive ones, packed into 32-bit words and read at once where
// they are aligned and all exist. Otherwise (rows that start anywhere) a word
// each, read one by one, kStride elements apart: neighbouring threads read
// neighbours. (Putting them together on arrival, kPack, waits for them: for
// kernels that have other warps to run and need the registers.)
template <class T, int V, bool kWide = true, int kStride = 1, bool kPack = false>
struct Raw {
  static constexpr bool kPacked = kWide || kPack;
  static constexpr int kWords = kPacked ? (V * (int)sizeof(T) + 3) / 4 : V;
  static_assert(!kWide || kStride == 1, "wide accesses are of consecutive elements");
  uint32_t w[kWords];

  static __device__ __forceinline__ uint32_t bits(const T* p) {
    if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const uint32_t*>(p));
    else return __ldg(reinterpret_cast<const unsigned short*>(p));
  }
  __device__ __forceinline__ float get(int k) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
    const uint32_t q = kPacked ? w[k / 2] : w[k];
    const bool high = kPacked && k % 2;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(high ? q & 0xFFFF0000u : q << 16);
    else
      return __half2float(__ushort_as_half((unsigned short)(high ? q >> 16 : q & 0xFFFFu)));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // whole: p is aligned to V elements, which all exist; otherwise the first
  // `have` do, the rest are zero.
  __device__ __forceinline__ void load(const T* p, bool whole, int have) {
    if constexpr (!kWide && kPack && sizeof(T) == 2) {
      if (have >= V) {
#pragma unroll
        for (int k = 0; k < V; k += 2)
          w[k / 2] = bits(p + k * kStride) | bits(p + (k + 1) * kStride) << 16;
      } else {
        zero();
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (k < have) w[k / 2] |= bits(p + k * kStride) << (k % 2 * 16);
      }
    } else if constexpr (!kWide) {
      if (have >= V) {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = bits(p + k * kStride);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = k < have ? bits(p + k * kStride) : 0;
      }
    } else if (whole) {
      if constexpr (V * sizeof(T) == 16) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
      } else if constexpr (V * sizeof(T) == 8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = q.x, w[1] = q.y;
      } else if constexpr (V * sizeof(T) == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else {
        w[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
      }
    } else {
      zero();
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (k < have) {
          if constexpr (sizeof(T) == 4) w[k] = bits(p + k);
          else w[k / 2] |= bits(p + k) << (k % 2 * 16);
        }
      }
    }
  }
};

// V float values from memory that the same kernel writes (no read-only path).
template <class T, int V, bool kWide, int kStride>
__device__ __forceinline__ void read_own(const T* p, bool whole, int have, float (&f)[V]) {
  if constexpr (kWide) {
    load_f32<T, V>(p, whole, have, f);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = k < have ? to_f32(p[k * kStride]) : 0.0f;
  }
}

// The same for a store of float values, rounded once.
template <class T, int V, bool kWide, int kStride>
__device__ __forceinline__ void store_raw(T* p, bool whole, int have, const float (&f)[V]) {
  if constexpr (kWide) {
    store_f32<T, V>(p, whole, have, f);
  } else if (have >= V) {
#pragma unroll
    for (int k = 0; k < V; ++k) p[k * kStride] = from_f32<T>(f[k]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (k < have) p[k * kStride] = from_f32<T>(f[k]);
  }
}

// i / d with the remainder in r, for i >= 0 and d > 0: in 32 bits where both
// fit, since a 64-bit division is about a hundred instructions (three of them
// took longer than all else of a single-token step).
__device__ __forceinline__ int64_t divide(int64_t i, int64_t d, int64_t& r) {
  if (((uint64_t)i | (uint64_t)d) >> 32 == 0) {
    const uint32_t q = (uint32_t)i / (uint32_t)d;
    r = (uint32_t)i - q * (uint32_t)d;
    return q;
  }
  const int64_t q = i / d;
  r = i - q * d;
  return q;
}

// An index of 4 or 8 bytes.
__device__ __forceinline__ int64_t load_index(const void* p, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(p)[i]
                    : (int64_t)static_cast<const int32_t*>(p)[i];
}

// Sequence b's length, clamped to [0, len].
__device__ __forceinline__ int64_t sequence_length(const void* lengths, int bytes, int64_t b,
                                                   int64_t len) {
  if (lengths == nullptr) return len;
  const int64_t n = load_index(lengths, bytes, b);
  return n < 0 ? 0 : n > len ? len : n;
}

// ------------------------------------------------------ nonlinearities
// 2^v, zero below 2^-126. The instruction's error is at most 1.4e-7 relative
// on [-20, 0], its mean -5e-9 near 0 and -5e-8 from -1 on (measured over 2^20
// points an interval).
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.44269504088896341f;

// 1 / v for v >= 1 (infinity gives 0); one unit of error.
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / (1 + exp(-v)); 0 and 1 in the limits.
__device__ __forceinline__ float sigmoid(float v) {
  return reciprocal(1.0f + exp2_fast(v * -kLog2e));
}

// ------------------------------------------------- pairs of binary32
// Two binary32 values in one 64-bit register pair, for the packed
// arithmetic (one issue for two operations; fma and mul are rounded to nearest
// one by one, for sums see add2).
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(F2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Not for products: given a packed product as an operand, a packed addition is
// joined with it into one rounding (nvcc 13.0, in spite of .rn and of
// --fmad=false), in some variants of a kernel and not in others.
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The same of any operands, as two single additions (the scan's gradient, 4 x 2048
// x 2048: 450 us with packed ones alone, 456 with these where products are
// summed, 468 with these alone).
__device__ __forceinline__ F2 add2_products(F2 a, F2 b) {
  float a0, a1, b0, b1;
  unpack2(a, a0, a1);
  unpack2(b, b0, b1);
  return pack2(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}

// softplus(v) = log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|), of two
// values. With s = e / (2 + e) <= 1/3, log1p(e) = 2 atanh(s) = 2 s (1 + s^2/3
// + s^4/5 + ...): seven terms leave (1/9)^7 / 15 = 1.4e-8 of the value, and
// the result keeps its relative accuracy where it is small (a few units of
// binary32).
__device__ __forceinline__ void softplus2(float& v0, float& v1) {
  const float e0 = exp2_fast(fabsf(v0) * -kLog2e), e1 = exp2_fast(fabsf(v1) * -kLog2e);
  const F2 s = mul2(pack2(e0, e1), pack2(reciprocal(2.0f + e0), reciprocal(2.0f + e1)));
  const F2 w = mul2(s, s);
  F2 p = pack2(1.0f / 13.0f, 1.0f / 13.0f);
  p = fma2(p, w, pack2(1.0f / 11.0f, 1.0f / 11.0f));
  p = fma2(p, w, pack2(1.0f / 9.0f, 1.0f / 9.0f));
  p = fma2(p, w, pack2(1.0f / 7.0f, 1.0f / 7.0f));
  p = fma2(p, w, pack2(1.0f / 5.0f, 1.0f / 5.0f));
  p = fma2(p, w, pack2(1.0f / 3.0f, 1.0f / 3.0f));
  p = fma2(p, w, pack2(1.0f, 1.0f));
  unpack2(fma2(mul2(s, pack2(2.0f, 2.0f)), p, pack2(fmaxf(v0, 0.0f), fmaxf(v1, 0.0f))), v0, v1);
}

__device__ __forceinline__ float softplus(float v) {
  float v1 = v;
  softplus2(v, v1);
  return v;
}

// ------------------------------------------------------------ host side
inline size_t model_esize(int dt) {
  switch (dt) {
    case CR_F32: return 4;
    case CR_BF16:
    case CR_F16: return 2;
    default: return 0;
  }
}

inline bool ptr_aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Whether rows of a (batch, time) strided tensor all start on `bytes`.
inline bool rows_aligned(const void* p, int64_t bs, int64_t ts, size_t es, size_t bytes) {
  return ptr_aligned(p, bytes) && ((size_t)bs * es) % bytes == 0 && ((size_t)ts * es) % bytes == 0;
}

// Whether an output pointer is one that the call reads (NULL: none).
inline bool overwrites(std::initializer_list<const void*> outs,
                       std::initializer_list<const void*> ins) {
  for (const void* o : outs)
    for (const void* i : ins)
      if (o != nullptr && o == i) return true;
  return false;
}

inline bool index_width_ok(int bytes) { return bytes == 4 || bytes == 8; }

inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxBlocks = 0x7FFFFFFF;  // of a grid's x axis

// A workspace begins with the status word of the calls that wait on the
// device (cr_sync_status); the model operators leave it as it is.
constexpr size_t kStatusBytes = 256;
inline char* past_status(void* ws) { return static_cast<char*>(ws) + kStatusBytes; }

}  // namespace cr

// Runs EXPR with T bound to the element type that DT names.
#define CR_MODEL_TYPE(DT, ...)                     \
  switch (DT) {                                    \
    case CR_F32: { using T = float; __VA_ARGS__; break; }          \
    case CR_BF16: { using T = __nv_bfloat16; __VA_ARGS__; break; } \
    default: { using T = __half; __VA_ARGS__; break; }             \
  }
