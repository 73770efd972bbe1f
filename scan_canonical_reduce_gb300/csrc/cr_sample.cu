// The next token of each row of logits: temperature, top-k, top-p, min-p.
//
// The row's tokens in the order of falling logits (equal ones by index) are
// kept up to a border, and the token is where the running sum of their weights
// w = 2^-y, y = (largest - logit) log2(e) / temperature, exceeds u times the
// kept sum. Sums are of integers in units of 2^-44, so that no order of
// summation changes them.
#include <cstdint>

#include "cr_device.cuh"
#include "cr_launch.h"
#include "cr_model.cuh"

namespace cr {
namespace {

constexpr int kSampleThreads = 1024;

// 2^(-j / 32) in units of 2^-63
__constant__ unsigned long long kRoots[32] = {
    0x8000000000000000ULL, 0x7D41D96DB915019DULL, 0x7A92BE8A92436616ULL, 0x77F25CCDEE6D7AE6ULL,
    0x75606373EE921C97ULL, 0x72DC8373BE41A454ULL, 0x70666F76154A7089ULL, 0x6DFDDBCBED791BABULL,
    0x6BA27E656B4EB57AULL, 0x69540EC8F895722DULL, 0x6712460A8FC24072ULL, 0x64DCDEC3371793D1ULL,
    0x62B39508AA836D6FULL, 0x6096266533384A2BULL, 0x5E8451CFAC061B5FULL, 0x5C7DD7A3B17DCF75ULL,
    0x5A827999FCEF3242ULL, 0x5891FAC0E95612C8ULL, 0x56AC1F752150A563ULL, 0x54D0AD5A753E077CULL,
    0x52FF6B54D8A89C75ULL, 0x513821818624B40CULL, 0x4F7A993048D088D7ULL, 0x4DC69CDCEAA72A9CULL,
    0x4C1BF828C6DC54B8ULL, 0x4A7A77D47F7B84B1ULL, 0x48E1E9B9D588E19BULL, 0x47521CC5A2E6A9E0ULL,
    0x45CAE0F1F545EB73ULL, 0x444C0740496D4294ULL, 0x42D561B3E6243D8AULL, 0x4166C34C5615D0ECULL};

struct Row {
  float top;     // the largest logit
  float ch, cl;  // log2(e) / temperature
};

// A logit as an unsigned number that falls as the logit rises; all ones for
// what is no candidate.
__device__ __forceinline__ uint32_t order_key(float l) {
  if (!(l > -INFINITY)) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 is 0
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}

// y in units of 2^-37 as (bin of 1/32, 32 bits of what is left); false where
// w < 2^-63.9.
__device__ __forceinline__ bool far_down(const Row& r, float l, int& bin, uint32_t& rest) {
  if (l == r.top) {
    bin = 0;
    rest = 0;
    return true;
  }
  const float s = r.top - l, bb = r.top - s, e = (r.top - (s + bb)) + (bb - l);
  const float yh = s * r.ch;
  if (!(yh < 63.9f)) return false;
  const float yl = fmaf(e, r.ch, fmaf(s, r.cl, fmaf(s, r.ch, -yh)));
  const float f = floorf(yh * 32.0f);
  const long long x = __float2ll_rn(fmaf(f, -0.03125f, yh) * 0x1p37f) +
                      __float2ll_rn(yl * 0x1p37f) + ((long long)f << 32);
  bin = (int)(x >> 32);
  rest = (uint32_t)x;
  return bin >= 0 ? true : (bin = 0, rest = 0, true);
}

// 1 - 2^-x in units of 2^-37 of x < 1/32 in units of 2^-37: z = x ln 2, 1 -
// exp(-z) = z - z^2 (1/2 - z (1/6 - z (1/24 - z / 120))), left out z^6 / 720 <
// 2^-42; what follows z is below 2^-12 and binary32 holds it to 2^-36.
__device__ __forceinline__ uint32_t one_minus(uint32_t rest) {
  const uint32_t z = __umulhi(rest, 0xB17217F8u);
  const float f = (float)z * 0x1p-37f;
  const float p = fmaf(-f, fmaf(-f, fmaf(-f, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f), 0.5f);
  return z - __float2uint_rn(f * f * p * 0x1p37f);
}

// w in units of 2^-44
__device__ __forceinline__ uint64_t weight(const Row& r, float l) {
  int bin;
  uint32_t rest;
  if (!far_down(r, l, bin, rest)) return 0;
  const uint64_t m = ((uint64_t)1 << 37) - one_minus(rest);
  const uint64_t w = __umul64hi(m << 26, kRoots[bin & 31]);  // units of 2^-62
  const int sh = 18 + (bin >> 5);
  return sh >= 64 ? 0 : (w + ((uint64_t)1 << (sh - 1))) >> sh;
}

template <class V>
__device__ V block_sum(V v, V* buf) {
#pragma unroll
  for (int s = 16; s > 0; s /= 2) v += __shfl_xor_sync(~0u, v, s);
  __syncthreads();
  if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
  __syncthreads();
  v = buf[threadIdx.x % 32];
#pragma unroll
  for (int s = 16; s > 0; s /= 2) v += __shfl_xor_sync(~0u, v, s);
  return v;
}

template <class T>
struct SampleIn {
  int64_t vocab;
  const T* logits;
  int64_t stride;
  const float* u;
  double temperature, top_p, min_p;
  int64_t top_k;
  const float *temperatures, *top_ps, *min_ps;
  const void* top_ks;
  int32_t index_bytes;
};

// A bisection over (key, index): the right answer, a pass over the row at a time.
template <class T>
__global__ void __launch_bounds__(kSampleThreads)
sample_kernel(SampleIn<T> in, int64_t* __restrict__ tokens) {
  __shared__ uint64_t buf[32];
  const int64_t row = blockIdx.x;
  const T* x = in.logits + row * in.stride;
  const int V = (int)in.vocab, tid = threadIdx.x;
  uint64_t least = ~0ull;  // the row's first, as (key, index)
  for (int i = tid; i < V; i += kSampleThreads) {
    const uint64_t k = (uint64_t)order_key(to_f32(x[i])) << 32 | (uint32_t)i;
    least = min(least, k);
  }
#pragma unroll
  for (int s = 16; s > 0; s /= 2) least = min(least, (uint64_t)__shfl_xor_sync(~0u, least, s));
  if (tid % 32 == 0) buf[tid / 32] = least;
  __syncthreads();
  least = buf[tid % 32];
#pragma unroll
  for (int s = 16; s > 0; s /= 2) least = min(least, (uint64_t)__shfl_xor_sync(~0u, least, s));
  const int first = (int)(uint32_t)least;
  const double temp = in.temperatures != nullptr ? in.temperatures[row] : in.temperature;
  if (least >> 32 == 0xFFFFFFFFu || !(temp > 0.0)) {
    if (tid == 0) tokens[row] = least >> 32 == 0xFFFFFFFFu ? -1 : first;
    return;
  }
  const double top_p = in.top_ps != nullptr ? in.top_ps[row] : in.top_p;
  const double min_p = in.min_ps != nullptr ? in.min_ps[row] : in.min_p;
  const int64_t top_k = in.top_ks != nullptr ? load_index(in.top_ks, in.index_bytes, row) : in.top_k;
  Row r;
  r.top = to_f32(x[first]) + 0.0f;
  const double c = fmin(1.4426950408889634 / temp, 1e37);
  r.ch = (float)c;
  r.cl = (float)(c - (double)r.ch);

  // what the tokens up to `to` sum up to: weights, or their number
  auto upto = [&](uint64_t to, bool count) {
    uint64_t s = 0;
    for (int i = tid; i < V; i += kSampleThreads) {
      const float l = to_f32(x[i]);
      const uint32_t key = order_key(l);
      if (key == 0xFFFFFFFFu || ((uint64_t)key << 32 | (uint32_t)i) > to) continue;
      s += count ? 1 : weight(r, l);
    }
    return block_sum(s, buf);
  };
  // the least (key, index) up to which they sum up to more than `target`
  auto search = [&](uint64_t target, uint64_t lo, uint64_t hi, bool count) {
    while (lo < hi) {
      const uint64_t mid = lo + (hi - lo) / 2;
      if (upto(mid, count) > target) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };
  uint64_t end = (uint64_t)0xFFFFFFFEu << 32 | 0xFFFFFFFFu;  // the last one kept
  if (top_k > 0 && top_k < V && upto(end, true) > (uint64_t)top_k)
    end = search((uint64_t)top_k - 1, least, end, true);
  uint64_t all = upto(end, false);
  if (top_p < 1.0) {
    const double t = ceil((top_p > 0.0 ? top_p : 0.0) * (double)all);
    // the first whose sum, itself included, reaches t
    if (t >= 1.0) end = search((uint64_t)t - 1, least, end, false);
    else end = least;
  }
  if (min_p > 0.0) {
    // w >= min_p: y <= -log2(min_p)
    const double y = fmax(-log2(min_p), 0.0) * 0x1p37;
    uint64_t n = 0;
    uint32_t worst = (uint32_t)(least >> 32);
    for (int i = tid; i < V; i += kSampleThreads) {
      const float l = to_f32(x[i]);
      int bin;
      uint32_t rest;
      if (order_key(l) == 0xFFFFFFFFu || !far_down(r, l, bin, rest)) continue;
      if ((double)((long long)bin << 32 | rest) <= y) worst = max(worst, order_key(l));
      ++n;
    }
    worst = __reduce_max_sync(~0u, worst);
    __syncthreads();
    if (tid % 32 == 0) buf[tid / 32] = worst;
    __syncthreads();
    worst = __reduce_max_sync(~0u, (uint32_t)buf[tid % 32]);
    __syncthreads();
    end = min(end, (uint64_t)worst << 32 | 0xFFFFFFFFu);
  }
  all = upto(end, false);
  const float u = in.u[row];
  const double at = (u > 0.0f ? fmin((double)u, 1.0 - 0x1p-24) : 0.0) * (double)all;
  const uint64_t got = search((uint64_t)at, least, end, false);
  if (tid == 0) tokens[row] = (int64_t)(uint32_t)got;
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
  if (a->vocab > (int64_t)1 << 20 || a->rows > kMaxBlocks) return CR_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CR_MODEL_TYPE(a->dt, {
    const SampleIn<T> in = {a->vocab, static_cast<const T*>(a->logits), a->row_stride, a->u,
                            a->temperature, a->top_p, a->min_p, a->top_k, a->temperatures,
                            a->top_ps, a->min_ps, a->top_ks, a->index_bytes};
    CR_LAUNCH(kKSample, s,
              sample_kernel<T><<<(unsigned)a->rows, kSampleThreads, 0, s>>>(in, tokens));
  });
  return cudaGetLastError() == cudaSuccess ? CR_OK : CR_ERR_CUDA;
}

}  // extern "C"
