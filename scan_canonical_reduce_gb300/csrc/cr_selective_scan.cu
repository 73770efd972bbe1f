// Selective state space scan and its single-token form (formulas in
// cr_selective_scan.cuh).
//
// The scan is bound by instruction issue and shared memory, not by DRAM: a
// channel step of 16 states is 16 exponentials and 64 multiply-adds against 8
// bytes in 16-bit types. Four lanes share a channel of 16 states (G = 4), four
// states each; the recurrence takes two steps at a time, whose exponents,
// inputs and outputs are pairs for the packed arithmetic. What belongs to a
// channel step alone (softplus, gate) is computed by one thread, a tile ahead
// of the recurrence or behind it. 8 x 1024 steps of 4096 channels, bf16: 186
// us, 1.4 TB/s.
#include "cr_selective_scan.cuh"

namespace cr {
namespace {

// Sequences with few channels are cut into segments that run side by side:
// a first launch (kStates) takes every segment but the last from a zero state
// to its end and its sum of delta, the second starts a segment from the
// state that these give, H' = exp(A sum delta) H + E in segment order. Every
// segment of the second launch reads the initial state, while the last one may
// be done: where the final state goes to the same place, the first launch
// leaves a copy for them.
struct Segments {
  int64_t count, len;
  float* E;        // [count - 1][batch][dim][NP]
  float* initial;  // [batch][dim][N], or NULL: no copy
  float* sum;      // [count - 1][batch][dim]
};

template <class T>
struct ScanOut {
  T* y;
  int64_t ybs, yts;
  float* final_state;
  float* checkpoints;
  int64_t n_check;
  bool wide_y, wide_check;
};

// Blocks an SM: 4 (126 registers) measured 396 us where 3 took 488 and 5 409
// (32,768 steps of 2048 channels, second launch).
#ifndef CR_SCAN_BLOCKS
#define CR_SCAN_BLOCKS 4
#endif
template <class T, int G, bool kStates, bool kWide>
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
        // a segment's growth or decay may leave the range that the states
        // stay in: then half of its exponent at a time (and so far that even
        // that leaves it, only a zero state stays finite)
        float a, a2;
        unpack2(A[k], a, a2);
        const float v = x * a;
        const bool far = fabsf(v) > 126.0f;
        const float f = exp2_fast(far ? fminf(0.5f * v, 127.0f) : v);
        h[k] = fmaf(f, far ? f * h[k] : h[k], e[k]);
      }
    }
  }

  using RowsE = Rows<T, VE, TL::NL, TL::ACC, TL::NV, kWide>;
  using RowsBC = Rows<T, kS, TL::NBC, TL::ACC_BC, G, kWide>;
  static_assert(kScanThreads % TL::NV == 0, "a thread's accesses are of one column");
  RowsE ru(in.u + b * in.ubs + d0, in.uts, begin, TL::TT, channels, kWide);
  RowsE rd(in.dt + b * in.dbs + d0, in.dts, begin, TL::TT, channels, kWide);
  RowsE rz(in.z + b * in.zbs + d0, in.zts, begin, TL::TT, channels, kWide);
  RowsBC rB(in.B + b * in.Bbs + group * in.N, in.Bts, begin, TL::TT, in.N, kWide);
  RowsBC rC(in.C + b * in.Cbs + group * in.N, in.Cts, begin, TL::TT, in.N, kWide);
  const bool gated = !kStates && in.z != nullptr;
  Raw<T, VE, kWide> pu[TL::NL][2], pd[TL::NL][2], pz[TL::NL][2];
  Raw<T, kS, kWide> pB[TL::NBC][2], pC[TL::NBC][2];
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
    Raw<T, VE, kWide> ku[TL::NL][2], kz[TL::NL][2];
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
      if (seg == 0 && sg.initial != nullptr) {
        const int64_t at = (b * in.dim + d) * in.N;
        load_states(in.state + at, n0, in.N, h);
        store_states(sg.initial + at, n0, in.N, false, h);
      }
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

// How a call's sequences are cut: a rule on sizes alone, so that results do not
// depend on the GPU. The first launch costs 0.6 of the second's time, so a
// call is cut only if it leaves schedulers without a warp (a GB300 has 608),
// into as many segments as give them four each, of a tile at least. Measured:
// 32,768 steps of 2048 channels (256 warps) 1,551 us whole, 611 us in nine
// segments; 4 x 2048 steps of 2048 channels (1024 warps) 150 us whole, 170 us
// in two.
#ifndef CR_SCAN_WARPS
#define CR_SCAN_WARPS 2432
#endif
#ifndef CR_SCAN_SPLIT_BELOW
#define CR_SCAN_SPLIT_BELOW 700
#endif
Segments scan_segments(int64_t batch, int64_t len, int64_t dim, int lanes) {
  constexpr int64_t kTile = 32;
  Segments sg;
  sg.E = sg.initial = sg.sum = nullptr;
  sg.count = 1;
  const int64_t warps = batch * ceil_div(dim * lanes, 32);
  if (warps < CR_SCAN_SPLIT_BELOW && warps > 0 && len >= 2 * kTile) {
    sg.count = CR_SCAN_WARPS / warps;
    const int64_t most = len / kTile;
    if (sg.count > most) sg.count = most;
    if (sg.count > 64) sg.count = 64;
  }
  sg.len = len > 0 ? ceil_div(ceil_div(len, sg.count), kTile) * kTile : kTile;
  sg.count = len > 0 ? ceil_div(len, sg.len) : 1;
  return sg;
}

// One token, bound by the state's traffic: 200 streams of 4096 channels and 16
// states take 22 us, 112 MB at 5.0 TB/s (with a thread for every four states,
// whose elementwise part is then done four times, 33 us). One stream of 2048
// channels 5 to 6 us with its call, 2.1 us of it on the device. A warp takes 32
// channels of a group: first a lane each, for delta, delta u and the gate, then
// G rounds of 32 / G channels by G lanes each, lane = c G + g, so that a
// round's states are consecutive in memory.
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
  const int lanes = scan_lanes(dstate);
  const int64_t segs = scan_segments(batch, len, dim, lanes).count;
  if (segs == 1) return kStatusBytes;
  return round256((size_t)batch * dim * (segs * lanes * kS + segs - 1) * 4) + kStatusBytes;
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
      (y == nullptr || (a->len > 1 && y_time_stride < a->dim) ||
       (a->batch > 1 && y_batch_stride < a->dim)))
    return CR_ERR_INVALID_ARG;
  const std::initializer_list<const void*> ins = {a->u, a->dt, a->z,       a->B,       a->C,
                                                  a->A, a->D,  a->dt_bias, a->lengths};
  if (a->batch > 0 && a->dim > 0 &&
      (overwrites({y, final_state, checkpoints}, ins) || overwrites({y, checkpoints}, {a->state})))
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
  if (sg.count > 1) {
    const int64_t states = a->batch * a->dim * lanes * kS;
    sg.E = reinterpret_cast<float*>(past_status(ws));
    if (a->state != nullptr && final_state == a->state) sg.initial = sg.E + (sg.count - 1) * states;
    sg.sum = sg.E + sg.count * states;
  }
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
    const bool wide_u = group_ok && rows_aligned(a->u, a->u_batch_stride, a->u_time_stride, es, bytes) &&
               rows_aligned(a->dt, a->dt_batch_stride, a->dt_time_stride, es, bytes) &&
               (a->z == nullptr ||
                rows_aligned(a->z, a->z_batch_stride, a->z_time_stride, es, bytes));
    out.wide_y = group_ok && rows_aligned(y, y_batch_stride, y_time_stride, es, bytes);
    out.wide_check = a->dstate % kS == 0 && ptr_aligned(checkpoints, 16);
    const bool wide_BC = a->dstate % kS == 0 &&
                         rows_aligned(a->B, a->B_batch_stride, a->B_time_stride, es, kS * es) &&
                         rows_aligned(a->C, a->C_batch_stride, a->C_time_stride, es, kS * es);
    const bool wide = wide_u && wide_BC;
    ScanIn<T> in = scan_in<T>(a);
    if (sg.count > 1)
      CR_LAUNCH(kKSelectiveScanStates, s,
                (wide ? selective_scan_kernel<T, G, true, true>
                      : selective_scan_kernel<T, G, true, false>)<<<(unsigned)(blocks * (sg.count - 1)), kScanThreads, 0, s>>>(in, out, sg));
    if (sg.initial != nullptr) in.state = sg.initial;
    CR_LAUNCH(kKSelectiveScan, s,
              (wide ? selective_scan_kernel<T, G, false, true>
                    : selective_scan_kernel<T, G, false, false>)<<<(unsigned)(blocks * sg.count), kScanThreads, 0, s>>>(in, out, sg));
  }));
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
  const std::initializer_list<const void*> ins = {a->u, a->dt, a->z,       a->B, a->C,
                                                  a->A, a->D,  a->dt_bias, slots};
  if (y == nullptr || (state == nullptr && state_rows > 0) ||
      (a->batch > 1 && y_batch_stride < a->dim) || overwrites({y, state}, ins) || y == state)
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
