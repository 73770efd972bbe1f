// Gradient of the selective state space scan (formulas in
// cr_selective_scan.cuh).
//
// Bound by latency at few warps: about 123 instructions a warp for a step of 8
// channels, a third of them for the sums of dB and dC over channels, issued in
// half of the cycles. 4 x 2048 steps of 2048 channels, 16 states, bf16: 442 us;
// its 256 blocks are 1.7 an SM, of the two that the registers of 16 steps of
// states allow.
#include "cr_selective_scan.cuh"

namespace cr {
namespace {

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
  bool wide_out, wide_check;
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

  static __device__ __forceinline__ F2 other(F2 send, int mask) {
    float a, b;
    unpack2(send, a, b);
    a = __shfl_xor_sync(~0u, a, mask);
    b = __shfl_xor_sync(~0u, b, mask);
    return pack2(a, b);
  }
  static __device__ __forceinline__ F2 exchange(F2 keep, F2 send, int mask) {
    return add2(keep, other(send, mask));
  }
  static __device__ __forceinline__ F2 first(F2 keep, F2 send) {  // of products
    return add2_products(keep, other(send, L / 2));
  }
  static __device__ __forceinline__ F2 select(bool s, F2 a, F2 b) { return s ? a : b; }

  // v[8] -> v[0 .. kPairs)
  static __device__ __forceinline__ void run(F2 (&v)[8], int c) {
    if (L >= 2) {  // slots {0, 1} or {2, 3}: v = B0 B1 C0 C1
      v[0] = first(v[0], v[2]);
      v[1] = first(v[1], v[3]);
      v[2] = first(v[4], v[6]);
      v[3] = first(v[5], v[7]);
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
// Two blocks an SM (235 registers); three spill and measured 609 us for 461.
// The last tile of a sequence that ends inside it has a copy of the adjoint
// loop that leaves out the steps past the end: selects within one loop would be
// 8 more instructions of some 250 for a pair of steps in every tile. (With the
// copy: no change at 16 states, 2 % more at 8.)
#ifndef CR_SCAN_BACK_BLOCKS
#define CR_SCAN_BACK_BLOCKS 2
#endif
template <class T, int G, bool kWide>
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

  using RowsE = Rows<T, VE, TL::NL, TL::ACC, TL::NV, kWide>;
  using RowsBC = Rows<T, kS, TL::NBC, TL::ACC_BC, G, kWide>;
  const int64_t last = (tiles - 1) * TT;
  RowsE ru(in.u + b * in.ubs + d0, in.uts, last, -TT, channels, kWide);
  RowsE rd(in.dt + b * in.dbs + d0, in.dts, last, -TT, channels, kWide);
  RowsE rz(in.z + b * in.zbs + d0, in.zts, last, -TT, channels, kWide);
  RowsE ry(o.dy + b * o.dybs + d0, o.dyts, last, -TT, channels, kWide);
  RowsBC rB(in.B + b * in.Bbs + group * in.N, in.Bts, last, -TT, in.N, kWide);
  RowsBC rC(in.C + b * in.Cbs + group * in.N, in.Cts, last, -TT, in.N, kWide);
  const bool gated = in.z != nullptr;
  Raw<T, VE, kWide> pu[TL::NL][2], pd[TL::NL][2], pz[TL::NL][2], py[TL::NL][2];
  Raw<T, kS, kWide> pB[TL::NBC][2], pC[TL::NBC][2];
  float next[kS] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto load = [&](int64_t tile) {
    const int left = (int)min(len - tile * TT, (int64_t)TT);
    ru.load(left, pu);
    rd.load(left, pd);
    if (gated) rz.load(left, pz);
    ry.load(left, py);
    rB.load(left, pB);
    rC.load(left, pC);
    // a lane without a channel holds none of another's states, which its own
    // decays could take out of range
    const float* q = o.checkpoints + ((b * o.n_check + tile) * in.dim + d) * in.N;
    if (live) read_states(q, n0, in.N, o.wide_check, next);
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
    Raw<T, VE, kWide> ku[TL::NL][2], kd[TL::NL][2], kz[TL::NL][2], ky[TL::NL][2];
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
    // past the sequence's end the state that q is a multiple of may have
    // overflowed, with nothing to multiply
    auto adjoint = [&](auto partial) {
      constexpr bool kPartial = decltype(partial)::value;
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
          const F2 gp = pack2(g0, g1);
          const F2 q = pack2(kPartial && t >= left ? 0.0f : r0 * h[t][k],
                             kPartial && t + 1 >= left ? 0.0f : r1 * h[t + 1][k]);
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
    };
    if (left == TT) adjoint(std::false_type{});
    else adjoint(std::true_type{});
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
      // past the sequence the terms are zero times a state, which may be infinite
      if (t >= len) s.x = 0.0f;
      if (t + 1 >= len) s.y = 0.0f;
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

}  // namespace
}  // namespace cr

extern "C" {

// Lanes that share a channel: those of its states, or more (whose states are
// zero) where the call has few warps, as each then walks its steps with less
// to do. A rule on sizes alone, so that results do not depend on the GPU; a
// GB300 has 608 schedulers, and 1,216 of these warps are resident. Gradient
// kernel, 4 states, 2048 steps, with 1, 2 and 4 lanes: 512 channels 529, 432
// and 364 us; 4 x 2048 channels (256 warps of one lane) 560, 514 and 493, with
// 2047 channels 1193, 610 and 551; 1024 steps of 8 x 2048 (512) 303, 282 and
// 494, of 16 x 2048 365, 556 and 981. 8 states, 4 x 2048 channels (512 warps
// of two lanes): 467 with 2, 492 with 4. 8 lanes lose from 512 channels up
// (16 states: 332 us with 4, 343 with 8).
static int backward_lanes(int64_t batch, int64_t dim, int dstate) {
  int lanes = cr::scan_lanes(dstate);
  while (lanes < 4) {
    const int64_t most = lanes == 1 ? 1216 : 608;  // warps with twice the lanes
    if (batch > most || dim > most * 32 || batch * cr::ceil_div(dim * lanes * 2, 32) > most) break;
    lanes *= 2;
  }
  return lanes;
}

// Blocks that share a group of a sequence: each leaves its own dB and dC.
static int64_t group_blocks(int64_t dim, int32_t groups, int lanes) {
  return cr::ceil_div(dim / groups, cr::kScanThreads / lanes);
}

size_t cr_selective_scan_backward_workspace_bytes(int64_t batch, int64_t len, int64_t dim,
                                                  int32_t dstate, int32_t groups) {
  using namespace cr;
  if (batch < 0 || len < 0 || dim < 0 || dstate < 1 || groups < 1 || dim % groups != 0) return 0;
  const int lanes = backward_lanes(batch, dim, dstate);
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
  if (a->dim == 0) {  // B and C are there all the same, and reach nothing
    const size_t bytes = (size_t)a->batch * a->len * a->groups * a->dstate * es;
    if (bytes == 0) return CR_OK;
    if (g->dB == nullptr || g->dC == nullptr || !ptr_aligned(g->dB, es) ||
        !ptr_aligned(g->dC, es) || overwrites({g->dB, g->dC}, {a->B, a->C}))
      return CR_ERR_INVALID_ARG;
    for (void* o : {g->dB, g->dC})
      if (cudaMemsetAsync(o, 0, bytes, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return CR_ERR_CUDA;
    return CR_OK;
  }
  if (g->dA == nullptr) return CR_ERR_INVALID_ARG;
  if (a->batch > 0 && a->len > 0 &&
      (g->dy == nullptr || g->checkpoints == nullptr || g->du == nullptr || g->ddt == nullptr ||
       g->dB == nullptr || g->dC == nullptr || (a->z != nullptr && g->dz == nullptr)))
    return CR_ERR_INVALID_ARG;
  const std::initializer_list<const void*> of_type = {g->du, g->ddt, g->dz, g->dB, g->dC};
  for (const void* o : of_type)
    if (!ptr_aligned(o, es)) return CR_ERR_INVALID_ARG;
  const std::initializer_list<const void*> ins = {
      a->u, a->dt,      a->z,     a->B,       a->C,  a->A,      a->D,
      a->dt_bias, a->state, a->lengths, g->dy, g->dfinal, g->checkpoints};
  if (overwrites(of_type, ins) || overwrites({g->dA, g->dD, g->ddt_bias, g->dstate}, ins))
    return CR_ERR_INVALID_ARG;
  if (!ptr_aligned(g->dy, es) || !ptr_aligned(g->dfinal, 4) || !ptr_aligned(g->checkpoints, 4) ||
      !ptr_aligned(g->dA, 4) || !ptr_aligned(g->dD, 4) || !ptr_aligned(g->ddt_bias, 4) ||
      !ptr_aligned(g->dstate, 4))
    return CR_ERR_INVALID_ARG;
  const size_t need = cr_selective_scan_backward_workspace_bytes(a->batch, a->len, a->dim,
                                                                 a->dstate, a->groups);
  if (ws == nullptr || !ptr_aligned(ws, 256) || ws_bytes < need) return CR_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int lanes = backward_lanes(a->batch, a->dim, a->dstate);
  const int64_t parts = group_blocks(a->dim, a->groups, lanes);
  const int64_t rows = a->batch * a->len * a->groups;
  const int64_t all = a->batch > 0 ? scan_blocks(a->batch, a->dim, a->groups, lanes) : 0;
  const int64_t sums = ceil_div(rows * 2 * a->dstate, kScanThreads);
  if ((a->batch > 0 && all == 0) || sums > kMaxBlocks) return CR_ERR_UNSUPPORTED;
  float* part_BC = reinterpret_cast<float*>(past_status(ws));
  float* part_A = reinterpret_cast<float*>(
      past_status(ws) + round256((size_t)rows * parts * 2 * (lanes * kS) * 4));
  if (a->batch > 0) {
    const unsigned blocks = (unsigned)all;
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
      const bool wide_u = group_ok && rows_aligned(a->u, a->u_batch_stride, a->u_time_stride, es, bytes) &&
               rows_aligned(a->dt, a->dt_batch_stride, a->dt_time_stride, es, bytes) &&
               rows_aligned(g->dy, g->dy_batch_stride, g->dy_time_stride, es, bytes) &&
               (a->z == nullptr ||
                rows_aligned(a->z, a->z_batch_stride, a->z_time_stride, es, bytes));
      o.wide_out = group_ok && rows_aligned(g->du, a->dim, a->dim, es, bytes) &&
                   rows_aligned(g->ddt, a->dim, a->dim, es, bytes) &&
                   rows_aligned(o.dz, a->dim, a->dim, es, bytes);
      const bool wide = wide_u && a->dstate % kS == 0 &&
                        rows_aligned(a->B, a->B_batch_stride, a->B_time_stride, es, kS * es) &&
                        rows_aligned(a->C, a->C_batch_stride, a->C_time_stride, es, kS * es);
      o.wide_check = a->dstate % kS == 0 && ptr_aligned(g->checkpoints, 16);
      CR_LAUNCH(kKSelectiveScanBackward, s,
                (wide ? selective_scan_backward_kernel<T, G, true>
                      : selective_scan_backward_kernel<T, G, false>)<<<blocks, kScanThreads, 0, s>>>(
                    scan_in<T>(a), o));
    }));
    if (cudaGetLastError() != cudaSuccess) return CR_ERR_CUDA;
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

}  // extern "C"
