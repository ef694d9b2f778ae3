// Selective scan with a decay per channel and state (the first-generation
// Mamba recurrence): for batch b, channel d of group g(d) and state n
//     delta = softplus(dt + dt_bias)
//     h[n]  = exp(delta A[d, n]) h[n] + delta x B[n]
//     y     = sum_n C[n] h[n] + D[d] x,   out = y silu(z)  (or y without z)
// and its backward.  With one decay per head a chunk turns into matrix products;
// with a decay per (d, n) there is no such product, and every (position, channel,
// state) costs one exponential and four operations of the FMA pipe: the
// arithmetic binds, not HBM (figures at each kernel).  An SM forms 32
// exponentials and issues 63 lanes of packed operations a clock, measured alone;
// loops of this mix, measured without any loads, reach 50 to 60 % of the issue
// slots, and so do these kernels.
//
// The sequence is cut into chunks that run in parallel, since B x channels
// alone leaves most of the machine idle:
//     k_sel_scan<.., false>  each chunk's state from zero, and the sum of its deltas
//     k_sel_combine          the state entering each chunk (decays exp(A sum delta))
//     k_sel_scan<.., true>   each chunk again from its state, with the outputs
// and in the backward
//     k_sel_state    the states as above and, for each group of chunks, the
//                    adjoint at its start, from zero after it:
//                    sum_t exp(A (delta_1 + .. + delta_t)) C_t dy_t
//     k_sel_combine  also the adjoint entering each group from the right
//     k_sel_bwd      the gradients of a group, chunk by chunk from its end
//     k_sel_bc, k_sel_params  fixed-order sums of dB, dC and of dA, dD, ddt_bias
// A lane owns two adjacent channels and SPT of their states, in registers; SL
// lanes share a channel's states where it has more, the other 32 / SL lane
// positions are channel pairs.  The arithmetic is in packed pairs (two states),
// so an element costs one exponential and two to three issues.
#include <cuda_bf16.h>

#include <type_traits>

#include "layer_math.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace lm;
using bf16 = __nv_bfloat16;

struct SelDims {
  int B, T, D, N, G, DG;  // DG: channels per group
  int L, nc;              // a block's positions, and how many such ranges
  int nh;                 // chunks with a state each (the backward has several a range)
  int ctiles;             // blocks' channel tiles per group
  int mode;               // how the rings copy (bytes: 16; 2: pairs; 1: elements)
  int v4;                 // state rows can be accessed 16 bytes at a time
  int wide;               // channel pairs can be read and written as one element
  int64_t zs, bs, cs;     // elements between positions of z, B, C
  int64_t zb, bb, cb;     // and between their batch rows
};

struct SelIn {
  const void *x, *dt;
  const float *dt_bias, *A;
  const void *B, *C;
  const float* D;
  const void* z;
  const int* lengths;
};

__device__ __forceinline__ int sel_len(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

__device__ __forceinline__ int64_t z_end(const SelDims& d) {  // elements from z's first to its last
  return (d.B - 1) * d.zb + (d.T - 1) * d.zs + d.D;
}

// A block's place: batch row, group of channels, chunk and first channel.
struct Place {
  int b, g, c, q0, ct;
};
__device__ __forceinline__ Place place(const SelDims& d, int channels) {
  Place p;
  int i = blockIdx.x;
  p.ct = i % d.ctiles;
  i /= d.ctiles;
  p.g = i % d.G;
  p.b = i / d.G;
  p.c = blockIdx.y;
  p.q0 = p.ct * channels;
  return p;
}

// A lane's channel pair.  Lanes past the group's channels (on false) are
// pointed at its first channel, so their loads stay in bounds; their results
// are not written.
struct Pair {
  int sl, cl, ch;  // state lane, channel lane, first channel
  bool on, two;
};
template <int SL>
__device__ __forceinline__ Pair lane_pair(const SelDims& d, const Place& p, int warp) {
  constexpr int CL = 32 / SL;
  Pair r;
  const int lane = threadIdx.x & 31;
  r.sl = lane / CL;
  r.cl = lane % CL;
  const int q = p.q0 + (warp * CL + r.cl) * 2;
  r.on = q < d.DG;
  r.two = q + 1 < d.DG;
  r.ch = p.g * d.DG + (r.on ? q : 0);
  return r;
}

constexpr float kLn2 = 0.6931471805599453f;

// B (and C) of one group in shared memory as fp32, NP states a position
// (zeros past N and past position n), TT positions at a time: fetched into
// registers while the tile before is used, then stored.
template <typename Tin, int NP, int TT, int NT>
struct RowTile {
  static constexpr int kPer = (TT * NP + NT - 1) / NT;
  Tin v[kPer];
  __device__ __forceinline__ void fetch(const Tin* src, int64_t stride, int N, int t0, int n) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x + i * NT, t = e / NP, k = e % NP;
      v[i] = (t < TT && k < N && t0 + t < n) ? src[(int64_t)(t0 + t) * stride + k] : from_f<Tin>(0.f);
    }
  }
  __device__ __forceinline__ void store(float* dst) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x + i * NT;
      if (e < TT * NP) dst[e] = to_f(v[i]);
    }
  }
};

__device__ __forceinline__ float2 lo2(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4& v) { return make_float2(v.z, v.w); }

// A warp's ring of its inputs: L positions of its channels for NI tensors a
// stage, S stages, filled by cp.async ahead of the computation (no registers
// held, and nothing the compiler can sink to the loads' use).  Where rows are
// 16-byte aligned a copy moves 16 bytes, else a pair of channels (4 or 8 bytes),
// or 4-byte elements.  ODD: bf16 rows that start in the middle of a 4-byte word
// at every other position are copied as the whole words that cover them, with
// the row's first channel at element 0 or 1 (plain loads, through registers, took
// three times as long over the whole scan).
constexpr int kStage = 8, kStages = 3;
constexpr int kU = 4;  // positions whose steps and gates are formed together

template <typename Tin, int CL, int NI, bool ODD, int L = kStage, int S = kStages>
struct Ring {
  static constexpr int CW = 2 * CL, W = CW + (ODD ? 8 : 0);  // channels; elements of a row
  static constexpr int kTensor = L * W, kOne = NI * kTensor;
  Tin* buf;
  const Tin* src[NI];  // position 0 of the range, the warp's first channel
  int64_t row[NI];     // elements between positions; NULL sources are skipped
  // ODD: the tensor's first element and its end, which no copy crosses
  const Tin *lo[ODD ? NI : 1], *hi[ODD ? NI : 1];
  int nt, nq, lane, mode;

  __device__ __forceinline__ void set(int i, const void* tensor, int64_t offset, int64_t stride,
                                      int64_t last) {
    const Tin* const t = static_cast<const Tin*>(tensor);
    src[i] = t ? t + offset : t;
    row[i] = stride;
    if constexpr (ODD) lo[i] = t, hi[i] = t + last;
  }
  // element of a row at which its first channel lies (t: from the range's start)
  __device__ __forceinline__ int shift(int i, int t) const {
    if constexpr (!ODD) return 0;
    return (int)((reinterpret_cast<uintptr_t>(src[i]) >> 1) + (uintptr_t)(t & (int)row[i])) & 1;
  }
  // stage s of the range into its slot; positions past nt, and channels past nq
  // are left as they are (their results are never written)
  __device__ __forceinline__ void fill(int s) {
    Tin* const dst0 = buf + (s % S) * kOne;
    const int t0 = s * L;
    if (t0 < nt) {
      if constexpr (ODD) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (!src[i]) continue;
          for (int e = lane; e < L * (CL + 1); e += 32) {  // a word each
            const int t = e / (CL + 1), c = (e % (CL + 1)) * 2, sh = shift(i, t0 + t);
            if (t0 + t >= nt || c >= min(CW, nq) + sh) continue;
            Tin* const dst = dst0 + i * kTensor + t * W + c;
            const Tin* const from = src[i] + (t0 + t) * row[i] + c - sh;
            if (from >= lo[i] && from + 2 <= hi[i]) {
              cp_async<4>(dst, from);
            } else {  // the tensor's first or last word
              if (from >= lo[i]) dst[0] = from[0];
              if (from + 1 >= lo[i] && from + 1 < hi[i]) dst[1] = from[1];
            }
          }
        }
      } else if (mode == 16) {
        constexpr int V = 16 / sizeof(Tin), R = CW / V;  // 16-byte pieces of a row
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (!src[i]) continue;
#pragma unroll
          for (int k = 0; k < (L * R + 31) / 32; ++k) {
            const int e = lane + 32 * k, t = e / R, c = (e % R) * V;
            if (e < L * R && t0 + t < nt && c < nq)
              cp_async<16>(dst0 + i * kTensor + t * W + c, src[i] + (t0 + t) * row[i] + c);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (!src[i]) continue;
          for (int e = lane; e < L * CL; e += 32) {
            const int t = e / CL, c = (e % CL) * 2;
            if (t0 + t >= nt || c >= nq) continue;
            Tin* dst = dst0 + i * kTensor + t * W + c;
            const Tin* from = src[i] + (t0 + t) * row[i] + c;
            if (mode == 2) {  // an aligned pair
              cp_async<2 * sizeof(Tin)>(dst, from);
            } else if constexpr (sizeof(Tin) == 4) {
              cp_async<4>(dst, from);
              if (c + 1 < nq) cp_async<4>(dst + 1, from + 1);
            }
          }
        }
      }
    }
    cp_commit();
  }
  // Makes stage s readable by the warp and starts the copy of stage s + S - 1
  // into the slot that every lane has left.
  __device__ __forceinline__ void next(int s) {
    cp_wait<S - 2>();
    __syncwarp();
    fill(s + S - 1);
  }
  __device__ __forceinline__ float2 get(int s, int t, int i, int cl) const {
    const Tin* const q = buf + (s % S) * kOne + i * kTensor + t * W + 2 * cl;
    if constexpr (ODD) {
      const int sh = shift(i, t + (L % 2 ? s * L : 0));
      return make_float2(to_f(q[sh]), to_f(q[sh + 1]));
    } else {
      return unpack2(*reinterpret_cast<const Two<Tin>*>(q));
    }
  }
};

// K2 pairs of a channel's states from s0 on (rows of N floats), 0 past N; as
// 16-byte accesses where rows allow (v4).
template <int K2>
__device__ __forceinline__ void ld_states(float2 (&v)[K2], const float* row, int s0, int N,
                                          bool on, bool v4) {
  if (v4) {
#pragma unroll
    for (int q = 0; q < K2 / 2; ++q) {
      const float4 f = on && s0 + 4 * q < N
                           ? *reinterpret_cast<const float4*>(row + s0 + 4 * q)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      v[2 * q] = lo2(f);
      v[2 * q + 1] = hi2(f);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K2; ++k) {
      const int s = s0 + 2 * k;
      v[k].x = on && s < N ? row[s] : 0.f;
      v[k].y = on && s + 1 < N ? row[s + 1] : 0.f;
    }
  }
}
template <int K2>
__device__ __forceinline__ void st_states(const float2 (&v)[K2], float* row, int s0, int N,
                                          bool v4) {
  if (v4) {
#pragma unroll
    for (int q = 0; q < K2 / 2; ++q)
      if (s0 + 4 * q < N)
        *reinterpret_cast<float4*>(row + s0 + 4 * q) =
            make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
  } else {
#pragma unroll
    for (int k = 0; k < K2; ++k) {
      const int s = s0 + 2 * k;
      if (s < N) row[s] = v[k].x;
      if (s + 1 < N) row[s + 1] = v[k].y;
    }
  }
}

constexpr int kFwdWarps = 4;
constexpr int kFwdBlocksPerSm = 3, kStateBlocksPerSm = 2;
constexpr int kFwdThreads = 32 * kFwdWarps;

template <typename Tin, int SPT, int SL, int NI, bool C, bool ODD>
struct PassSmem {
  static constexpr int NP = SPT * SL, TT = NP > 16 ? 512 / NP : 32;
  float B[2][TT * NP], Cm[2][C ? TT * NP : 4];
  __align__(16) Tin ring[kFwdWarps][kStages * Ring<Tin, 32 / SL, NI, ODD>::kOne];
};

// Forward pass over one chunk.  OUT: with the outputs, from the state
// hin (B, nc, D, N) (or init when there is one chunk); else the chunk's state
// from zero into hin and its delta sum into sumd (B, nc, D).
// Without OUT it is bound by the exponentials (61 to 65 % of their unit's slots,
// 59 % of the issue slots): 82 us for 4 x 4096 x 1536 x 16 elements and 374 us for
// 65536 x 2048 x 16, 5.0 and 5.7 elements a ps.  With OUT (the product with C, the
// gate, the store) by issue: 58 %, 50 % of the exponentials' slots; 116 and 550 us.
// Where few warps are resident (short inputs) each waits for its own chain, about 4
// clocks an instruction, so ranges are cut short there.
template <typename Tin, typename Tout, int SPT, int SL, bool OUT, bool ODD>
__global__ void __launch_bounds__(kFwdThreads, kFwdBlocksPerSm)
    k_sel_scan(SelIn in, const float* __restrict__ init, float* __restrict__ hin,
               float* __restrict__ sumd, Tout* __restrict__ out, float* __restrict__ final_state,
               SelDims d) {
  constexpr int CL = 32 / SL, NP = SPT * SL, K2 = SPT / 2, NI = OUT ? 3 : 2;
  using Smem = PassSmem<Tin, SPT, SL, NI, OUT, ODD>;
  constexpr int TT = Smem::TT;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem);
  griddep_launch_dependents();
  if (d.nc > 1 && OUT) griddep_wait();
  const int warp = threadIdx.x >> 5;
  const Place p = place(d, CL * 2 * kFwdWarps);
  const Pair ln = lane_pair<SL>(d, p, warp);
  const int n = sel_len(in.lengths, p.b, d.T);
  const int t0 = p.c * d.L, t1 = min(d.T, t0 + d.L), nt = max(min(t1, n) - t0, 0);
  const int64_t row0 = (int64_t)p.b * d.T + t0;
  const int qw = p.q0 + warp * CL * 2, cw = p.g * d.DG + qw;  // the warp's first channel
  const bool gated = OUT && in.z;
  const Tin* Bm = static_cast<const Tin*>(in.B) + p.b * d.bb + t0 * d.bs + (int64_t)p.g * d.N;
  const Tin* Cm = static_cast<const Tin*>(in.C) + p.b * d.cb + t0 * d.cs + (int64_t)p.g * d.N;
  Ring<Tin, CL, NI, ODD> ring;
  ring.buf = sm.ring[warp];
  const int64_t all = (int64_t)d.B * d.T * d.D;
  ring.set(0, in.x, row0 * d.D + cw, d.D, all);
  ring.set(1, in.dt, row0 * d.D + cw, d.D, all);
  if constexpr (OUT) ring.set(2, in.z, p.b * d.zb + t0 * d.zs + cw, d.zs, z_end(d));
  ring.nt = nt, ring.nq = d.DG - qw, ring.lane = threadIdx.x & 31, ring.mode = d.mode;
  ring.fill(0);
  ring.fill(1);
  RowTile<Tin, NP, TT, kFwdThreads> tB, tC;
  tB.fetch(Bm, d.bs, d.N, 0, nt);
  if (OUT) tC.fetch(Cm, d.cs, d.N, 0, nt);

  float2 a2[2][K2], h[2][K2], bias = f2(0.f), skip = f2(0.f), sd = f2(0.f);
  if (in.dt_bias) bias = make_float2(in.dt_bias[ln.ch], in.dt_bias[ln.ch + (ln.two ? 1 : 0)]);
  if (OUT && in.D) skip = make_float2(in.D[ln.ch], in.D[ln.ch + (ln.two ? 1 : 0)]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bool on = j ? ln.two : ln.on;
    const int ch = ln.ch + j;
    const float* h0 = nullptr;
    if (OUT && on) {
      if (d.nc > 1)
        h0 = hin + (((int64_t)p.b * d.nc + p.c) * d.D + ch) * d.N;
      else if (init)
        h0 = init + ((int64_t)p.b * d.D + ch) * d.N;
    }
    ld_states<K2>(a2[j], in.A + (int64_t)ch * d.N, ln.sl * SPT, d.N, on, d.v4);
    ld_states<K2>(h[j], h0, ln.sl * SPT, d.N, h0 != nullptr, d.v4);
#pragma unroll
    for (int k = 0; k < K2; ++k) a2[j][k] = mul2(a2[j][k], f2(kLog2e));
  }
  tB.store(sm.B[0]);
  if (OUT) tC.store(sm.Cm[0]);
  __syncthreads();
  Tout* o = OUT ? out + row0 * d.D + ln.ch : nullptr;
  int buf = 0;
  for (int tb = 0; tb < nt; tb += TT) {
    const bool more = tb + TT < nt;
    if (more) {
      tB.fetch(Bm, d.bs, d.N, tb + TT, nt);
      if (OUT) tC.fetch(Cm, d.cs, d.N, tb + TT, nt);
    }
    const int te = min(TT, nt - tb);
    for (int ts = 0; ts < te; ts += kStage) {
      const int stage = (tb + ts) / kStage;
      ring.next(stage);
#pragma unroll 1
      for (int tu = 0; tu < kStage; tu += kU) {
        if (ts + tu >= te) break;
        float2 xv[kU], dl[kU], gate[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          gate[u] = f2(1.f);
          xv[u] = ring.get(stage, tu + u, 0, ln.cl);
          dl[u] = softplus2(add2(ring.get(stage, tu + u, 1, ln.cl), bias));
          if constexpr (OUT)
            if (gated) {
              const float2 zv = ring.get(stage, tu + u, 2, ln.cl);
              gate[u] = mul2(zv, sigmoid2(zv));
            }
        }
        auto step = [&](int u) {
          const int t = ts + tu + u;
          const float4* Bv = reinterpret_cast<const float4*>(sm.B[buf] + t * NP + ln.sl * SPT);
          const float4* Cv = reinterpret_cast<const float4*>(sm.Cm[buf] + t * NP + ln.sl * SPT);
          const float2 dtx = mul2(dl[u], xv[u]);
          if (!OUT) sd = add2(sd, dl[u]);
          float2 y[2] = {f2(0.f), f2(0.f)};
#pragma unroll
          for (int q = 0; q < SPT / 4; ++q) {
            const float4 b4 = Bv[q];
            float4 c4;
            if (OUT) c4 = Cv[q];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int k = 2 * q + i;
              const float2 bk = i ? hi2(b4) : lo2(b4);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 a = decay2(j ? dl[u].y : dl[u].x, a2[j][k]);
                h[j][k] = fma2(a, h[j][k], mul2(f2(j ? dtx.y : dtx.x), bk));
                if (OUT) y[j] = fma2(h[j][k], i ? hi2(c4) : lo2(c4), y[j]);
              }
            }
          }
          if (OUT) {
            float2 yv = make_float2(y[0].x + y[0].y, y[1].x + y[1].y);
#pragma unroll
            for (int w = CL; w < 32; w <<= 1) {
              yv.x += __shfl_xor_sync(0xffffffffu, yv.x, w);
              yv.y += __shfl_xor_sync(0xffffffffu, yv.y, w);
            }
            yv = fma2(skip, xv[u], yv);
            if (gated) yv = mul2(yv, gate[u]);
            if (ln.on && ln.sl == 0) st_two(o, yv, ln.two, d.wide);
            o += d.D;
          }
        };
        if (ts + tu + kU <= te) {  // no branch between the steps: they overlap
#pragma unroll
          for (int u = 0; u < kU; ++u) step(u);
        } else {
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (ts + tu + u < te) step(u);
        }
      }
    }
    if (more) {
      buf ^= 1;
      tB.store(sm.B[buf]);
      if (OUT) tC.store(sm.Cm[buf]);
      __syncthreads();
    }
  }
  if (!ln.on) return;
  if (OUT && ln.sl == 0)
    for (int t = nt; t < t1 - t0; ++t, o += d.D) st_two(o, f2(0.f), ln.two, d.wide);
  if (!OUT && ln.sl == 0) {
    float* s = sumd + ((int64_t)p.b * d.nc + p.c) * d.D + ln.ch;
    s[0] = sd.x;
    if (ln.two) s[1] = sd.y;
  }
  if (OUT && (!final_state || p.c != d.nc - 1)) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (j && !ln.two) break;
    float* v = OUT ? final_state + ((int64_t)p.b * d.D + ln.ch + j) * d.N
                   : hin + (((int64_t)p.b * d.nc + p.c) * d.D + ln.ch + j) * d.N;
    st_states<K2>(h[j], v, ln.sl * SPT, d.N, d.v4);
  }
}

constexpr int kBwdL = 32;  // positions of a backward chunk

// The backward's first pass over a group of chunks: each chunk's state from zero
// (hin) and delta sum, and the group's adjoint at its start from zero after it
// (gin).  Running products of the decays give the adjoint in the forward
// direction, from the same exponentials.  159 us for 4 x 4096 x 1536 x 16 (2.5
// elements a ps) at 248 registers, two blocks an SM: issue, 48 % of the slots.
template <typename Tin, int SPT, int SL, bool ODD>
__global__ void __launch_bounds__(kFwdThreads, kStateBlocksPerSm)
    k_sel_state(SelIn in, const Tin* __restrict__ dout, float* __restrict__ hin,
                float* __restrict__ gin, float* __restrict__ sumd, float* __restrict__ sumg,
                SelDims d) {
  constexpr int CL = 32 / SL, NP = SPT * SL, K2 = SPT / 2;
  using Smem = PassSmem<Tin, SPT, SL, 4, true, ODD>;
  constexpr int TT = Smem::TT;
  static_assert(kBwdL % TT == 0, "a chunk is whole tiles");
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem);
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const Place p = place(d, CL * 2 * kFwdWarps);
  const Pair ln = lane_pair<SL>(d, p, warp);
  const int n = sel_len(in.lengths, p.b, d.T);
  const int t0 = p.c * d.L, t1 = min(d.T, t0 + d.L), nt = max(min(t1, n) - t0, 0);
  const int64_t row0 = (int64_t)p.b * d.T + t0;
  const int qw = p.q0 + warp * CL * 2, cw = p.g * d.DG + qw;
  const Tin* Bm = static_cast<const Tin*>(in.B) + p.b * d.bb + t0 * d.bs + (int64_t)p.g * d.N;
  const Tin* Cm = static_cast<const Tin*>(in.C) + p.b * d.cb + t0 * d.cs + (int64_t)p.g * d.N;
  Ring<Tin, CL, 4, ODD> ring;
  ring.buf = sm.ring[warp];
  const int64_t all = (int64_t)d.B * d.T * d.D;
  ring.set(0, in.x, row0 * d.D + cw, d.D, all);
  ring.set(1, in.dt, row0 * d.D + cw, d.D, all);
  ring.set(2, dout, row0 * d.D + cw, d.D, all);
  ring.set(3, in.z, p.b * d.zb + t0 * d.zs + cw, d.zs, z_end(d));
  ring.nt = nt, ring.nq = d.DG - qw, ring.lane = threadIdx.x & 31, ring.mode = d.mode;
  ring.fill(0);
  ring.fill(1);
  RowTile<Tin, NP, TT, kFwdThreads> tB, tC;
  tB.fetch(Bm, d.bs, d.N, 0, nt);
  tC.fetch(Cm, d.cs, d.N, 0, nt);

  float2 a2[2][K2], h[2][K2], pr[2][K2], gl[2][K2], bias = f2(0.f), sd = f2(0.f), sg = f2(0.f);
  if (in.dt_bias) bias = make_float2(in.dt_bias[ln.ch], in.dt_bias[ln.ch + (ln.two ? 1 : 0)]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    ld_states<K2>(a2[j], in.A + (int64_t)(ln.ch + j) * d.N, ln.sl * SPT, d.N, j ? ln.two : ln.on,
                  d.v4);
#pragma unroll
    for (int k = 0; k < K2; ++k) {
      a2[j][k] = mul2(a2[j][k], f2(kLog2e));
      h[j][k] = gl[j][k] = f2(0.f);
      pr[j][k] = f2(1.f);
    }
  }
  auto write = [&](float* dst, int64_t at, float2 (&v)[2][K2]) {  // at: row of (.., D)
    if (!ln.on) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j && !ln.two) break;
      st_states<K2>(v[j], dst + (at * d.D + ln.ch + j) * d.N, ln.sl * SPT, d.N, d.v4);
    }
  };
  auto write_sum = [&](float* dst, int64_t at, float2 v) {
    if (!ln.on || ln.sl != 0) return;
    dst[at * d.D + ln.ch] = v.x;
    if (ln.two) dst[at * d.D + ln.ch + 1] = v.y;
  };
  tB.store(sm.B[0]);
  tC.store(sm.Cm[0]);
  __syncthreads();
  int buf = 0;
  const int64_t c0 = (int64_t)p.b * d.nh + t0 / kBwdL;  // the range's first chunk
  for (int tb = 0; tb < t1 - t0; tb += TT) {
    const bool more = tb + TT < nt;
    if (more) {
      tB.fetch(Bm, d.bs, d.N, tb + TT, nt);
      tC.fetch(Cm, d.cs, d.N, tb + TT, nt);
    }
    const int te = min(TT, nt - tb);
    for (int ts = 0; ts < te; ts += kStage) {
      const int stage = (tb + ts) / kStage;
      ring.next(stage);
#pragma unroll 1
      for (int tu = 0; tu < kStage; tu += kU) {
        if (ts + tu >= te) break;
        float2 xv[kU], dl[kU], dy[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          xv[u] = ring.get(stage, tu + u, 0, ln.cl);
          dl[u] = softplus2(add2(ring.get(stage, tu + u, 1, ln.cl), bias));
          dy[u] = ring.get(stage, tu + u, 2, ln.cl);
          if (in.z) {
            const float2 zv = ring.get(stage, tu + u, 3, ln.cl);
            dy[u] = mul2(dy[u], mul2(zv, sigmoid2(zv)));
          }
        }
        auto step = [&](int u) {
          const int t = ts + tu + u;
          const float4* Bv = reinterpret_cast<const float4*>(sm.B[buf] + t * NP + ln.sl * SPT);
          const float4* Cv = reinterpret_cast<const float4*>(sm.Cm[buf] + t * NP + ln.sl * SPT);
          const float2 dtx = mul2(dl[u], xv[u]);
          sd = add2(sd, dl[u]);
#pragma unroll
          for (int q = 0; q < SPT / 4; ++q) {
            const float4 b4 = Bv[q], c4 = Cv[q];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int k = 2 * q + i;
              const float2 bk = i ? hi2(b4) : lo2(b4), ck = i ? hi2(c4) : lo2(c4);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 a = decay2(j ? dl[u].y : dl[u].x, a2[j][k]);
                h[j][k] = fma2(a, h[j][k], mul2(f2(j ? dtx.y : dtx.x), bk));
                pr[j][k] = mul2(pr[j][k], a);
                gl[j][k] = fma2(pr[j][k], mul2(f2(j ? dy[u].y : dy[u].x), ck), gl[j][k]);
              }
            }
          }
        };
        if (ts + tu + kU <= te) {  // no branch between the steps: they overlap
#pragma unroll
          for (int u = 0; u < kU; ++u) step(u);
        } else {
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (ts + tu + u < te) step(u);
        }
      }
    }
    if ((tb + TT) % kBwdL == 0 || tb + TT >= t1 - t0) {  // a chunk ends
      const int64_t at = c0 + tb / kBwdL;
      write(hin, at, h);
      write_sum(sumd, at, sd);
      sg = add2(sg, sd);
      sd = f2(0.f);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < K2; ++k) h[j][k] = f2(0.f);
    }
    if (more) {
      buf ^= 1;
      tB.store(sm.B[buf]);
      tC.store(sm.Cm[buf]);
      __syncthreads();
    }
  }
  write(gin, (int64_t)p.b * d.nc + p.c, gl);
  write_sum(sumg, (int64_t)p.b * d.nc + p.c, sg);
}

// hin (B, nh, D, N): each chunk's own state -> the state entering it, in place:
// H_{c+1} = exp(A sumd_c) H_c + S_c.  With gin (blockIdx.y = 1; B, nc, D, N): each
// range's own adjoint at its start -> the adjoint entering it from the right:
// G_c = gin_c + exp(A sumg_c) G_{c+1}.  One thread per (b, d, n); the next kC
// chunks are loaded while the chain runs over kC.  (The last own value of either
// walk is not needed.)  Bound by the loads' latency: 8 us for the forward of
// 4 x 4096 x 1536 x 16, 30 for the backward, which has a state every 32 positions.
__global__ void __launch_bounds__(256)
    k_sel_combine(const float* __restrict__ A, const float* __restrict__ init,
                  const float* __restrict__ dfinal, float* __restrict__ hin,
                  float* __restrict__ gin, const float* __restrict__ sumd,
                  const float* __restrict__ sumg, SelDims d) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t DN = (int64_t)d.D * d.N, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= d.B * DN) return;
  const int b = (int)(i / DN);
  const int64_t dn = i - b * DN;
  const float a2 = A[dn] * kLog2e;
  const bool rev = blockIdx.y == 1;
  const int nc = rev ? d.nc : d.nh;
  const int64_t sv = rev ? -DN : DN, ss = rev ? -d.D : d.D;
  float* v = (rev ? gin : hin) + ((int64_t)b * nc + (rev ? nc - 1 : 0)) * DN + dn;
  const float* sm = (rev ? sumg : sumd) + ((int64_t)b * nc + (rev ? nc - 1 : 0)) * d.D + dn / d.N;
  const float* start = rev ? dfinal : init;
  float acc = start ? start[i] : 0.f;
  constexpr int kC = 8;
  float e[kC], o[kC], ne[kC], no[kC];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int u = 0; u < kC; ++u) {
      const bool in = c0 + u < nc - 1;
      no[u] = in ? v[(c0 + u) * sv] : 0.f;
      ne[u] = in ? sm[(c0 + u) * ss] : 0.f;
    }
  };
  fetch(0);
  for (int c0 = 0; c0 < nc; c0 += kC) {
#pragma unroll
    for (int u = 0; u < kC; ++u) e[u] = ne[u], o[u] = no[u];
    fetch(c0 + kC);
#pragma unroll
    for (int u = 0; u < kC; ++u)
      if (c0 + u < nc) {
        v[(c0 + u) * sv] = acc;
        acc = fmaf(decay(e[u], a2), acc, o[u]);
      }
  }
}

// Sums v[0 .. NV) over CL lanes cl.  Halving exchanges: at each step a lane
// keeps one half of the values and sends the other to the lane that keeps that
// one, so lane cl ends with the totals [cl * NV / CL, (cl + 1) * NV / CL) in
// v[0 ..]; with fewer values than lanes, CL / NV consecutive lanes end with the
// total cl / (CL / NV).
template <int NV, int CL>
__device__ __forceinline__ void reduce_lanes(float (&v)[NV], int cl) {
  int half = NV / 2;
#pragma unroll
  for (int o = CL / 2; o > 0; o >>= 1) {
    if (half > 0) {
      const bool up = (cl & o) != 0;
#pragma unroll
      for (int i = 0; i < NV / 2; ++i)
        if (i < half) {
          const float send = up ? v[i] : v[i + half];
          const float keep = up ? v[i + half] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      half /= 2;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
}

// 1 - e^-v for v >= 0: by its series to v^7 below 1/4 (the next term is under
// 2e-9 of it), where the difference would cancel.
__device__ __forceinline__ float one_minus_exp(float v) {
  float p = fmaf(v, 1.f / 5040.f, -1.f / 720.f);
  p = fmaf(p, v, 1.f / 120.f);
  p = fmaf(p, v, -1.f / 24.f);
  p = fmaf(p, v, 1.f / 6.f);
  p = fmaf(p, v, -0.5f);
  p = fmaf(p, v, 1.f);
  return v < 0.25f ? p * v : 1.f - ex2(-v * kLog2e);
}

constexpr int kBwdTS = 4, kBwdWarps = 4, kBwdThreads = 32 * kBwdWarps;
constexpr int kBwdTiles = kBwdL / kBwdTS;

// The next chunk's inputs are copied over the kept states once those are used
// up: x, dt, dout and z where they fit (z is else read when it is needed).
template <typename Tin, int SPT, int SL, bool ODD>
struct BwdSmem {
  static constexpr int NP = SPT * SL, CL = 32 / SL, Q = SPT / 4;
  static constexpr int NI = sizeof(Tin) == 2 || Q == 1 ? 4 : 3;
  float B[kBwdL * NP], C[kBwdL * NP];
  float red[2][kBwdWarps][kBwdTS][2 * NP];
  float2 delta[kBwdWarps][kBwdL][CL], x[kBwdWarps][kBwdL][CL], dy[kBwdWarps][kBwdL][CL];
  using R = Ring<Tin, CL, NI, ODD, kBwdL, 1>;
  union {
    float4 start[kBwdTiles - 1][2][Q][32];
    __align__(16) unsigned char raw[R::kOne * sizeof(Tin)];
  } w[kBwdWarps];
};

// Gradients of a group of chunks, from its last chunk to its first.  With the
// state that enters a chunk known, the warp walks forward once, keeping the
// state at every kBwdTS-th position, then backward tile by tile: the tile's
// states are formed again into registers, and at each position
//     g = C dy + a_next g_next,  w = (a g) h_prev
//     dA += delta w,  ddelta = sum_n (A w + x g B),  dx = delta sum_n g B + D dy
//     dB_t += delta x g,  dC_t += dy h   (sums over the group's channels).
// The last two are sums over lanes by halving exchanges, one exchange a value.
// The first exchange needs no selects: a lane in the upper half of the channel
// lanes holds its two groups of four states in the other order, so what it
// keeps and what it sends sit in the same registers in every lane.  The
// block's warps are then added in shared memory, and each block writes its
// part (B, T, G, ctiles, 2 N).
// 578 us for 4 x 4096 x 1536 x 16 (0.7 elements a ps): 27 instructions an element,
// of which the two walks forward are 8 and the sums over lanes 4, at 50 % of the
// issue slots with 236 registers a thread.  Measured and not kept: tiles of 2
// positions, chunks of 16 (580 to 628, and combine 38 -> 97 us), half the states a
// lane on twice the warps.  h_prev is formed again rather than taken from
// a h_prev = h - delta x B, which cancels where the decay is strong.
template <typename Tin, typename Tout, int SPT, int SL, bool ODD>
__global__ void __launch_bounds__(kBwdThreads, 2)
    k_sel_bwd(SelIn in, const Tin* __restrict__ dout, const float* __restrict__ hin,
              const float* __restrict__ gin, Tout* __restrict__ dx, Tout* __restrict__ ddt,
              Tout* __restrict__ dz, float* __restrict__ bcpart, float* __restrict__ dApart,
              float* __restrict__ ppart, float* __restrict__ dinit, SelDims d) {
  constexpr int CL = 32 / SL, NP = SPT * SL, K2 = SPT / 2, Q = SPT / 4;
  static_assert(SL >= 2 && Q <= 2, "a lane finishes one of its two channels");
  extern __shared__ __align__(16) unsigned char raw_smem[];
  using Smem = BwdSmem<Tin, SPT, SL, ODD>;
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem);
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place(d, CL * 2 * kBwdWarps);
  const Pair ln = lane_pair<SL>(d, p, warp);
  const int sl = ln.sl, cl = ln.cl;
  const int swap = Q == 2 && cl >= CL / 2 ? 1 : 0;  // order of the state groups
  const int n = sel_len(in.lengths, p.b, d.T);
  const int64_t rowb = (int64_t)p.b * d.T;
  const Tin* x = static_cast<const Tin*>(in.x) + rowb * d.D;
  const Tin* dt = static_cast<const Tin*>(in.dt) + rowb * d.D;
  const Tin* z = in.z ? static_cast<const Tin*>(in.z) + p.b * d.zb : nullptr;
  const Tin* Bm = static_cast<const Tin*>(in.B) + p.b * d.bb + (int64_t)p.g * d.N;
  const Tin* Cm = static_cast<const Tin*>(in.C) + p.b * d.cb + (int64_t)p.g * d.N;
  const Tin* const dout0 = dout;
  dout += rowb * d.D;

  // the channel that this lane finishes: the pair's first or second
  const int fj = sl & 1, fch = ln.ch + fj;
  const bool fon = sl < 2 && (fj ? ln.two : ln.on);
  const float fskip = in.D && fon ? in.D[fch] : 0.f;
  float2 bias = f2(0.f);
  if (in.dt_bias) bias = make_float2(in.dt_bias[ln.ch], in.dt_bias[ln.ch + (ln.two ? 1 : 0)]);

  // register pair k of a lane: states st(k), st(k) + 1
  auto st = [&](int k) { return sl * SPT + ((k >> 1) ^ swap) * 4 + (k & 1) * 2; };
  float2 a2[2][K2], h[2][K2], gc[2][K2], dA[2][K2];
  const int64_t gat = ((int64_t)p.b * d.nc + p.c) * d.D + ln.ch;  // row of (B, nc, D)
  auto load = [&](float2 (&v)[2][K2], const float* rows) {  // the pair's rows of states
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        float2 g[2];
        ld_states<2>(g, rows + (int64_t)j * d.N, st(2 * q), d.N, j ? ln.two : ln.on, d.v4);
        v[j][2 * q] = g[0];
        v[j][2 * q + 1] = g[1];
      }
  };
  load(a2, in.A + (int64_t)ln.ch * d.N);
  load(gc, gin + gat * d.N);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int k = 0; k < K2; ++k) {
      a2[j][k] = mul2(a2[j][k], f2(kLog2e));
      dA[j][k] = f2(0.f);
    }
  // starts the copy of chunk c's inputs (positions and channels past the end are
  // left as they are: they are masked when they are read)
  const int qw = p.q0 + warp * CL * 2, cw = p.g * d.DG + qw;
  auto ring_of = [&](int c) {
    typename Smem::R r;
    const int64_t t0 = (int64_t)c * kBwdL, at = (rowb + t0) * d.D + cw;
    const int64_t all = (int64_t)d.B * d.T * d.D;
    r.buf = reinterpret_cast<Tin*>(sm.w[warp].raw);
    r.set(0, in.x, at, d.D, all);
    r.set(1, in.dt, at, d.D, all);
    r.set(2, dout0, at, d.D, all);
    if constexpr (Smem::NI == 4) r.set(3, in.z, p.b * d.zb + t0 * d.zs + cw, d.zs, z_end(d));
    r.nt = max(n - (int)t0, 0), r.nq = d.DG - qw, r.lane = lane, r.mode = d.mode;
    return r;
  };
  float dD = 0.f, dbias = 0.f;
  int ph = 0;
  // this thread's element of a tile's dB / dC sums (position u, state e)
  constexpr int kSum = kBwdTS * 2 * NP, kSums = (kSum + kBwdThreads - 1) / kBwdThreads;
  const int cfirst = p.c * (d.L / kBwdL), clast = min(d.nh, cfirst + d.L / kBwdL) - 1;
  for (int c = clast; c >= cfirst; --c) {
    const int t0 = c * kBwdL, t1 = min(d.T, t0 + kBwdL), nt = max(min(t1, n) - t0, 0);
    float cD = 0.f, cbias = 0.f;  // the chunk's parts: shorter sums round less
    const auto raw = ring_of(c);
    if (c == clast) ring_of(c).fill(0);
    const int64_t hat = ((int64_t)p.b * d.nh + c) * d.D + ln.ch;
    auto enter = [&]() { load(h, hin + hat * d.N); };  // the state entering the chunk
    __syncthreads();  // the chunk after this one is done with B and C
    {
      RowTile<Tin, NP, kBwdL, kBwdThreads> tB, tC;
      tB.fetch(Bm + t0 * d.bs, d.bs, d.N, 0, nt);
      tC.fetch(Cm + t0 * d.cs, d.cs, d.N, 0, nt);
      enter();
      cp_wait<0>();
      __syncwarp();
      // lane -> (position sl + SL i, pair cl): delta, x and dy, once
#pragma unroll 4
      for (int t = sl; t < kBwdL; t += SL) {
        float2 xv = raw.get(0, t, 0, cl);
        float2 dl = softplus2(add2(raw.get(0, t, 1, cl), bias));
        float2 dy = raw.get(0, t, 2, cl);
        if (z) {
          float2 zv;
          if constexpr (Smem::NI == 4)
            zv = raw.get(0, t, 3, cl);
          else
            zv = unpack2(ld_two(z + (int64_t)(t0 + max(min(t, nt - 1), 0)) * d.zs + ln.ch, ln.two,
                                d.wide));
          dy = mul2(dy, mul2(zv, sigmoid2(zv)));
        }
        if (!ln.on || t >= nt) dl = xv = dy = f2(0.f);
        if (!ln.two) dl.y = xv.y = dy.y = 0.f;
        sm.delta[warp][t][cl] = dl;
        sm.x[warp][t][cl] = xv;
        sm.dy[warp][t][cl] = dy;
      }
      tB.store(sm.B);
      tC.store(sm.C);
    }
    __syncthreads();
    const float4* const sBv = reinterpret_cast<const float4*>(sm.B);
    const float4* const sCv = reinterpret_cast<const float4*>(sm.C);
    auto at4 = [&](int t, int q) { return (t * NP + sl * SPT) / 4 + (q ^ swap); };
    auto step = [&](int t) {  // h at position t from h at t - 1
      const float2 dl = sm.delta[warp][t][cl], xd = mul2(dl, sm.x[warp][t][cl]);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float4 b4 = sBv[at4(t, q)];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int k = 2 * q + i;
            const float2 a = decay2(j ? dl.y : dl.x, a2[j][k]);
            h[j][k] = fma2(a, h[j][k], mul2(f2(j ? xd.y : xd.x), i ? hi2(b4) : lo2(b4)));
          }
      }
    };
    for (int tile = 1; tile < kBwdTiles; ++tile) {
#pragma unroll
      for (int u = 0; u < kBwdTS; ++u) step((tile - 1) * kBwdTS + u);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          sm.w[warp].start[tile - 1][j][q][lane] =
              make_float4(h[j][2 * q].x, h[j][2 * q].y, h[j][2 * q + 1].x, h[j][2 * q + 1].y);
    }
    for (int tile = kBwdTiles - 1; tile >= 0; --tile) {
      const int tb = tile * kBwdTS;
      if (tile == 0 && c > cfirst) {  // the kept states are used up
        __syncwarp();
        ring_of(c - 1).fill(0);
      }
      auto begin = [&]() {  // h = the state entering the tile
        if (tile == 0) {
          enter();
          return;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const float4 v = sm.w[warp].start[tile - 1][j][q][lane];
            h[j][2 * q] = lo2(v);
            h[j][2 * q + 1] = hi2(v);
          }
      };
      // a lane's pair of sums -> the sum of the channel it finishes, over its SL lanes
      auto finish = [&](float2 v) {
        float r = (fj ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, fj ? v.x : v.y, CL);
#pragma unroll
        for (int o = 2 * CL; o < 32; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        return r;
      };
      float2 hs[kBwdTS][2][K2];
      float ys[kBwdTS];  // sum_n C h of the channel that this lane finishes
      begin();
#pragma unroll
      for (int u = 0; u < kBwdTS; ++u) {
        step(tb + u);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < K2; ++k) hs[u][j][k] = h[j][k];
        if (z) {
          float2 y[2] = {f2(0.f), f2(0.f)};
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const float4 c4 = sCv[at4(tb + u, q)];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              y[j] = fma2(h[j][2 * q], lo2(c4), y[j]);
              y[j] = fma2(h[j][2 * q + 1], hi2(c4), y[j]);
            }
          }
          ys[u] = finish(make_float2(y[0].x + y[0].y, y[1].x + y[1].y));
        }
      }
      begin();
#pragma unroll
      for (int u = kBwdTS - 1; u >= 0; --u) {
        const int t = tb + u;
        const float2 dl = sm.delta[warp][t][cl], xv = sm.x[warp][t][cl], dy = sm.dy[warp][t][cl];
        const float2 xd = mul2(dl, xv);
        float2 gb[2] = {f2(0.f), f2(0.f)}, aw[2] = {f2(0.f), f2(0.f)}, vB[K2], vC[K2];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const float4 b4 = sBv[at4(t, q)], c4 = sCv[at4(t, q)];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int k = 2 * q + i;
            const float2 bk = i ? hi2(b4) : lo2(b4), ck = i ? hi2(c4) : lo2(c4);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 dlj = f2(j ? dl.y : dl.x);
              const float2 g = fma2(ck, f2(j ? dy.y : dy.x), gc[j][k]);
              gc[j][k] = mul2(decay2(dlj.x, a2[j][k]), g);
              const float2 w = mul2(gc[j][k], u > 0 ? hs[u > 0 ? u - 1 : 0][j][k] : h[j][k]);
              dA[j][k] = fma2(dlj, w, dA[j][k]);
              aw[j] = fma2(a2[j][k], w, aw[j]);
              gb[j] = fma2(g, bk, gb[j]);
              if (j == 0) {
                vB[k] = mul2(f2(xd.x), g);
                vC[k] = mul2(f2(dy.x), hs[u][0][k]);
              } else {
                vB[k] = fma2(f2(xd.y), g, vB[k]);
                vC[k] = fma2(f2(dy.y), hs[u][1][k], vC[k]);
              }
            }
          }
        }
        float v[8];  // four states of dB and of dC
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (Q == 2) {
            const float2 ob = make_float2(__shfl_xor_sync(0xffffffffu, vB[2 + i].x, CL / 2),
                                          __shfl_xor_sync(0xffffffffu, vB[2 + i].y, CL / 2));
            const float2 oc = make_float2(__shfl_xor_sync(0xffffffffu, vC[2 + i].x, CL / 2),
                                          __shfl_xor_sync(0xffffffffu, vC[2 + i].y, CL / 2));
            vB[i] = add2(vB[i], ob);
            vC[i] = add2(vC[i], oc);
          }
          v[2 * i] = vB[i].x, v[2 * i + 1] = vB[i].y;
          v[4 + 2 * i] = vC[i].x, v[4 + 2 * i + 1] = vC[i].y;
        }
        constexpr int RL = Q == 2 ? CL / 2 : CL;  // lanes left to add over
        reduce_lanes<8, RL>(v, cl % RL);
        constexpr int kPer = 8 > RL ? 8 / RL : 1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int e = (cl % RL) * 8 / RL + i;  // < 4: dB, else dC
          sm.red[ph][warp][u][(e >> 2) * NP + sl * SPT + swap * 4 + (e & 3)] = v[i];
        }
        const float fgb = finish(make_float2(gb[0].x + gb[0].y, gb[1].x + gb[1].y));
        const float faw = finish(make_float2(aw[0].x + aw[0].y, aw[1].x + aw[1].y)) * kLn2;
        const float fdl = fj ? dl.y : dl.x, fdy = fj ? dy.y : dy.x, fx = fj ? xv.y : xv.x;
        // sigmoid(v) = 1 - e^-softplus(v)
        const float dv = t < nt ? fmaf(fx, fgb, faw) * one_minus_exp(fdl) : 0.f;
        if (fon && t < t1 - t0) {
          const int64_t at = (rowb + t0 + t) * d.D + fch;
          dx[at] = from_f<Tout>(fmaf(fdl, fgb, fskip * fdy));
          ddt[at] = from_f<Tout>(dv);
          cD = fmaf(fdy, fx, cD);
          cbias += dv;
          if (z) ys[u] = fmaf(fskip, fx, ys[u]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSums; ++k) {
        const int i = threadIdx.x + k * kBwdThreads;
        const int u = i / (2 * NP), e = i % (2 * NP), st = e % NP;
        if ((kSum % kBwdThreads == 0 || i < kSum) && st < d.N && tb + u < t1 - t0) {
          float a = 0.f;
#pragma unroll
          for (int wv = 0; wv < kBwdWarps; ++wv) a += sm.red[ph][wv][u][e];
          bcpart[(((rowb + t0 + tb + u) * d.G + p.g) * d.ctiles + p.ct) * (2 * d.N) +
                 (e / NP) * d.N + st] = a;
        }
      }
      if (z && fon) {  // the tile's dy is used up: its slots take y for dz
#pragma unroll
        for (int u = 0; u < kBwdTS; ++u)
          reinterpret_cast<float*>(&sm.dy[warp][tb + u][cl])[fj] = ys[u];
      }
      ph ^= 1;
    }
    dD += cD;
    dbias += cbias;
    if (z) {  // dz = dout y silu'(z), a pair a lane
      __syncwarp();
      constexpr int kE = 8;
      for (int i0 = 0; i0 < kBwdL / SL; i0 += kE) {
        Two<Tin> rg[kE], rz[kE];
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          const int64_t t = t0 + max(min(sl + SL * (i0 + i), nt - 1), 0);
          rg[i] = ld_two(dout + t * d.D + ln.ch, ln.two, d.wide);
          rz[i] = ld_two(z + t * d.zs + ln.ch, ln.two, d.wide);
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          const int t = sl + SL * (i0 + i);
          if (i0 + i < kBwdL / SL && ln.on && t < t1 - t0) {
            const float2 zv = unpack2(rz[i]), sg = sigmoid2(zv);
            const float2 ds = fma2(mul2(sg, zv), fma2(sg, f2(-1.f), f2(1.f)), sg);
            const float2 o = mul2(mul2(unpack2(rg[i]), sm.dy[warp][t][cl]), ds);
            st_two(dz + (rowb + t0 + t) * d.D + ln.ch, t < nt ? o : f2(0.f), ln.two, d.wide);
          }
        }
      }
    }
  }
  if (fon) {
    const int64_t at = ((int64_t)p.b * d.nc + p.c) * d.D + fch;
    ppart[at * 2] = dD;
    ppart[at * 2 + 1] = dbias;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (!(j ? ln.two : ln.on)) continue;
    float* gi = dinit && p.c == 0 ? dinit + ((int64_t)p.b * d.D + ln.ch + j) * d.N : nullptr;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float2 a[2] = {dA[j][2 * q], dA[j][2 * q + 1]}, g[2] = {gc[j][2 * q], gc[j][2 * q + 1]};
      st_states<2>(a, dApart + (gat + j) * d.N, st(2 * q), d.N, d.v4);
      if (gi) st_states<2>(g, gi, st(2 * q), d.N, d.v4);
    }
  }
}

// dB, dC (B, T, G, N): the channel tiles' parts, in order.
__global__ void __launch_bounds__(256)
    k_sel_bc(const float* __restrict__ part, float* __restrict__ dB, float* __restrict__ dC,
             int64_t rows, int ctiles, int N) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rows * 2 * N) return;
  const int64_t r = i / (2 * N);
  const int e = (int)(i - r * 2 * N);
  const float* p = part + r * ctiles * 2 * N + e;
  float a = 0.f;
  for (int c = 0; c < ctiles; ++c) a += p[(int64_t)c * 2 * N];
  if (e < N)
    dB[r * N + e] = a;
  else
    dC[r * N + e - N] = a;
}

// dA (D, N), dD and ddt_bias (D): the (batch, chunk) parts, a block per 32
// entries, its 8 warps taking every 8th part.
__global__ void __launch_bounds__(256)
    k_sel_params(const float* __restrict__ dApart, const float* __restrict__ ppart,
                 float* __restrict__ dA, float* __restrict__ dD, float* __restrict__ dbias,
                 int parts, int64_t DN, int D, int blocksA) {
  __shared__ float red[8][32];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool isA = (int)blockIdx.x < blocksA;
  const int64_t w = isA ? DN : 2 * (int64_t)D;
  const int64_t i = (int64_t)(isA ? blockIdx.x : blockIdx.x - blocksA) * 32 + lane;
  const float* p = isA ? dApart : ppart;
  float a = 0.f;
  if (i < w)
    for (int k = warp; k < parts; k += 8) a += p[k * w + i];
  red[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && i < w) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][lane];
    if (isA)
      dA[i] = s;
    else if (i & 1) {
      if (dbias) dbias[i >> 1] = s;
    } else if (dD) {
      dD[i >> 1] = s;
    }
  }
}

// ------------------------------------------------------------------- host

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int sel_dims(const ssd_selective_shape* s, SelDims* d) {
  if (!s || s->batch < 1 || s->seqlen < 1 || s->channels < 1 || s->dstate < 1 || s->ngroups < 1 ||
      s->channels % s->ngroups != 0)
    return SSD_ERR_INVALID_ARG;
  if ((s->in_dtype != SSD_F32 && s->in_dtype != SSD_BF16) ||
      (s->out_dtype != SSD_F32 && s->out_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  const int64_t gn = s->ngroups * s->dstate;
  if ((s->z_row_stride && s->z_row_stride < s->channels) ||
      (s->b_row_stride && s->b_row_stride < gn) || (s->c_row_stride && s->c_row_stride < gn) ||
      s->z_batch_stride < 0 || s->b_batch_stride < 0 || s->c_batch_stride < 0)
    return SSD_ERR_INVALID_ARG;
  if (s->in_dtype == SSD_F32 && s->out_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->dstate > 64 || s->batch >= 65536 || s->seqlen >= (1 << 30) || s->channels >= (1 << 24))
    return SSD_ERR_UNSUPPORTED;
  d->B = (int)s->batch, d->T = (int)s->seqlen, d->D = (int)s->channels, d->N = (int)s->dstate;
  d->G = (int)s->ngroups, d->DG = d->D / d->G;
  d->zs = s->z_row_stride ? s->z_row_stride : d->D;
  d->bs = s->b_row_stride ? s->b_row_stride : gn;
  d->cs = s->c_row_stride ? s->c_row_stride : gn;
  d->zb = s->z_row_stride ? s->z_batch_stride : d->zs * d->T;
  d->bb = s->b_row_stride ? s->b_batch_stride : d->bs * d->T;
  d->cb = s->c_row_stride ? s->c_batch_stride : d->cs * d->T;
  return SSD_OK;
}

// Forward ranges of whole stages: as many as fill the machine once
// (kFwdBlocksPerSm blocks an SM); one (no state pass) where the channels fill half
// of it by themselves (2048 positions of 30 x 2048 channels: 715 us, 943 in two
// ranges; of 27 x 2048, which do not: 715 and 732), or up to kOneRange positions
// (1536 channels: 16 positions in one range take 10.3 us, in ranges of a stage 12.6;
// 24 12.4 and 12.4; 32 14.4 and 12.4).  Short ranges pay where the machine is not
// full: 4 x 333 x 300 takes 22.6 us, 26.7 with ranges of 16 positions, 36.9 with 32.
constexpr int kOneRange = 24;
int fwd_chunks(SelDims* d) {
  const int sl = d->N > 32 ? 4 : d->N > 16 ? 2 : 1;
  d->ctiles = ceil_div(d->DG, 32 / sl * 2 * kFwdWarps);
  const int64_t blocks = (int64_t)d->B * d->G * d->ctiles;
  int64_t nc = kFwdBlocksPerSm * 152 / blocks;
  if (nc < 2 || d->T <= kOneRange) nc = 1;
  d->L = ceil_div(ceil_div(d->T, nc), kStage) * kStage;
  d->nc = d->nh = ceil_div(d->T, d->L);
  return blocks <= 0x7fffffff ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

// Backward: the two passes have their own channel tiles (first: as the
// forward; main: half the states a lane).  Ranges of whole chunks; their length
// is the one with the shortest modelled time: each pass runs in waves of its
// two blocks an SM, and a range costs the main pass about 24 issues an element,
// the first 7.  Ranges of twice and of half that length: forward and backward of
// 4 x 4096 x 1536 x 16 take 960 us (1009, 968), of 8192 x 1024 x 16 378 (614, 399).
// A range has at most kMaxPer chunks and a grid kMaxGridY rows of blocks, a range each,
// so a sequence has at most kMaxPer * kMaxGridY chunks.
constexpr int kMaxPer = 64, kMaxGridY = 65535;
int bwd_main_tiles(const SelDims& d) {
  const int sl = d.N > 32 ? 8 : d.N > 16 ? 4 : 2;
  return ceil_div(d.DG, 32 / sl * 2 * kBwdWarps);
}
int bwd_chunks(SelDims* d) {
  const int sl = d->N > 32 ? 4 : d->N > 16 ? 2 : 1;
  d->ctiles = ceil_div(d->DG, 32 / sl * 2 * kFwdWarps);
  d->nh = ceil_div(d->T, kBwdL);
  const int64_t bg = (int64_t)d->B * d->G, wave = 2 * 152;
  int64_t best = -1;
  int best_per = 1;
  for (int per = 1; per <= d->nh && per <= kMaxPer; ++per) {
    const int64_t nc = ceil_div(d->nh, per);
    if (nc > kMaxGridY) continue;
    const int64_t main = (bg * bwd_main_tiles(*d) * nc + wave - 1) / wave;
    const int64_t wave1 = kStateBlocksPerSm * 152;
    const int64_t first = (bg * d->ctiles * nc + wave1 - 1) / wave1;
    // (half a chunk's time for what a range costs by itself)
    const int64_t cost = (24 * main + 7 * first) * (2 * per + 1);
    if (best < 0 || cost < best) best = cost, best_per = per;
  }
  if (best < 0 || bg * d->ctiles > 0x7fffffff || bg * bwd_main_tiles(*d) > 0x7fffffff ||
      (int64_t)d->B * d->T * d->G > ((int64_t)1 << 31))
    return SSD_ERR_UNSUPPORTED;
  d->L = best_per * kBwdL;
  d->nc = ceil_div(d->nh, best_per);
  return SSD_OK;
}

struct SelBwdWs {
  float *hin, *gin, *sumd, *sumg, *bc, *dA, *pp;
  size_t total;
};

SelBwdWs bwd_ws(const SelDims& d, void* base) {
  SelBwdWs w;
  size_t off = 0;
  auto take = [&](size_t n) {
    float* p = reinterpret_cast<float*>(static_cast<char*>(base) + off);
    off = align_up(off + n * sizeof(float), 256);
    return p;
  };
  const size_t cd = (size_t)d.B * d.nc * d.D, hd = (size_t)d.B * d.nh * d.D;
  w.hin = take(hd * d.N);
  w.gin = take(cd * d.N);
  w.sumd = take(hd);
  w.sumg = take(cd);
  w.dA = take(cd * d.N);
  w.pp = take(cd * 2);
  w.bc = take((size_t)d.B * d.T * d.G * bwd_main_tiles(d) * 2 * d.N);
  w.total = off;
  return w;
}

dim3 sel_grid(const SelDims& d, int chunks) {
  return dim3((unsigned)((int64_t)d.B * d.G * d.ctiles), chunks);
}

cudaError_t combine(const SelDims& d, const float* A, const float* init, const float* dfinal,
                    float* hin, float* gin, const float* sumd, const float* sumg, cudaStream_t s) {
  const int64_t n = (int64_t)d.B * d.D * d.N;
  const dim3 grid((unsigned)((n + 255) / 256), gin ? 2 : 1);
  cudaError_t e;
  SSD_LAUNCH("k_sel_combine", s, e = launch_pdl(k_sel_combine, grid, 256, 0, s, A, init, dfinal,
                                                hin, gin, sumd, sumg, d));
  return e;
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return bytes <= 48 * 1024
             ? cudaSuccess
             : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename Tin, typename Tout, int SPT, int SL, bool ODD>
int sel_forward(const SelDims& d, const SelIn& in, const float* init, void* out, float* fin,
                float* hin, float* sumd, cudaStream_t s) {
  Tout* const o = static_cast<Tout*>(out);
  auto kstate = k_sel_scan<Tin, Tout, SPT, SL, false, ODD>;
  auto kout = k_sel_scan<Tin, Tout, SPT, SL, true, ODD>;
  constexpr size_t ms = sizeof(PassSmem<Tin, SPT, SL, 2, false, ODD>);
  constexpr size_t mo = sizeof(PassSmem<Tin, SPT, SL, 3, true, ODD>);
  if (allow_smem(kstate, ms) != cudaSuccess || allow_smem(kout, mo) != cudaSuccess)
    return SSD_ERR_CUDA;
  if (d.nc > 1) {
    SSD_LAUNCH("k_sel_chunk_state", s,
               kstate<<<sel_grid(d, d.nc - 1), kFwdThreads, ms, s>>>(in, nullptr, hin, sumd,
                                                                     nullptr, nullptr, d));
    if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;  // no states to go on from
    if (combine(d, in.A, init, nullptr, hin, nullptr, sumd, nullptr, s) != cudaSuccess)
      return SSD_ERR_CUDA;
    cudaError_t e;
    SSD_LAUNCH("k_sel_scan", s, e = launch_pdl(kout, sel_grid(d, d.nc), kFwdThreads, mo, s, in,
                                               init, hin, sumd, o, fin, d));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
  }
  SSD_LAUNCH("k_sel_scan", s,
             kout<<<sel_grid(d, 1), kFwdThreads, mo, s>>>(in, init, hin, sumd, o, fin, d));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

struct SelGrads {
  void *dx, *ddt;
  float *dA, *dB, *dC, *dD;
  void* dz;
  float *ddt_bias, *dinit;
};

// SPT, SL: the first pass's states and state lanes; the main pass has half the
// states a lane (its live set is three times as large) on twice the lanes.
template <typename Tin, typename Tout, int SPT, int SL, bool ODD>
int sel_backward(const SelDims& d, const SelIn& in, const float* init, const void* dout,
                 const float* dfinal, const SelGrads& g, const SelBwdWs& w, cudaStream_t s) {
  const Tin* go = static_cast<const Tin*>(dout);
  auto kstate = k_sel_state<Tin, SPT, SL, ODD>;
  constexpr size_t ms = sizeof(PassSmem<Tin, SPT, SL, 4, true, ODD>);
  if (allow_smem(kstate, ms) != cudaSuccess) return SSD_ERR_CUDA;
  SSD_LAUNCH("k_sel_state", s, kstate<<<sel_grid(d, d.nc), kFwdThreads, ms, s>>>(
                                   in, go, w.hin, w.gin, w.sumd, w.sumg, d));
  if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;  // no states to go on from
  if (combine(d, in.A, init, dfinal, w.hin, w.gin, w.sumd, w.sumg, s) != cudaSuccess)
    return SSD_ERR_CUDA;
  SelDims m = d;
  m.ctiles = bwd_main_tiles(d);
  auto kern = k_sel_bwd<Tin, Tout, SPT / 2, SL * 2, ODD>;
  constexpr size_t smem = sizeof(BwdSmem<Tin, SPT / 2, SL * 2, ODD>);
  if (allow_smem(kern, smem) != cudaSuccess) return SSD_ERR_CUDA;
  cudaError_t e;
  SSD_LAUNCH("k_sel_bwd", s,
             e = launch_pdl(kern, sel_grid(m, m.nc), kBwdThreads, smem, s, in, go, w.hin, w.gin,
                            static_cast<Tout*>(g.dx), static_cast<Tout*>(g.ddt),
                            static_cast<Tout*>(g.dz), w.bc, w.dA, w.pp, g.dinit, m));
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  const int64_t rows = (int64_t)d.B * d.T * d.G, DN = (int64_t)d.D * d.N;
  SSD_LAUNCH("k_sel_bc", s,
             e = launch_pdl(k_sel_bc, (unsigned)((rows * 2 * d.N + 255) / 256), 256, 0, s, w.bc,
                            g.dB, g.dC, rows, m.ctiles, d.N));
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  const int ba = ceil_div(DN, 32), bp = ceil_div(2 * (int64_t)d.D, 32);
  SSD_LAUNCH("k_sel_params", s,
             e = launch_pdl(k_sel_params, ba + bp, 256, 0, s, w.dA, w.pp, g.dA, g.dD, g.ddt_bias,
                            d.B * d.nc, DN, d.D, ba));
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// The instantiation for a state count and a pair of types.
template <int V>
using Int = std::integral_constant<int, V>;
template <typename F>
int by_states(int N, F&& f) {
  if (N <= 8) return f(Int<8>{}, Int<1>{});
  if (N <= 16) return f(Int<16>{}, Int<1>{});
  if (N <= 32) return f(Int<16>{}, Int<2>{});
  return f(Int<16>{}, Int<4>{});
}

// How the inputs (and outputs of oe bytes an element) can be accessed: the
// rings' mode, the pairs' width, and the state rows.
void access(SelDims* d, int ie, int oe, const void* const* ins, const void* const* outs,
            const void* z, const void* const* states) {
  d->v4 = 1;
  for (int i = 0; i < 3; ++i) d->v4 = d->v4 && vec_ok(states[i], d->N, 4, 4);
  auto rows_ok = [&](int v) {
    bool ok = d->DG % v == 0;
    for (int i = 0; i < 3; ++i) ok = ok && vec_ok(ins[i], d->D, ie, v);
    return ok && (!z || (vec_ok(z, d->zs, ie, v) && vec_ok(z, d->zb, ie, v)));
  };
  d->mode = rows_ok(16 / ie) ? 16 : rows_ok(2) ? 2 : 1;
  d->wide = d->mode != 1;
  for (int i = 0; i < 3; ++i) d->wide = d->wide && vec_ok(outs[i], d->D, oe, 2);
}

bool off(const void* p, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(esize - 1)) != 0;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_selective_scan_fwd_workspace_size(const ssd_selective_shape* shape) {
  SelDims d;
  if (sel_dims(shape, &d) != SSD_OK || fwd_chunks(&d) != SSD_OK) return 0;
  if (d.nc == 1) return 256;
  const size_t cd = (size_t)d.B * d.nc * d.D;
  return align_up(cd * d.N * sizeof(float), 256) + align_up(cd * sizeof(float), 256);
}

size_t ssd_selective_scan_bwd_workspace_size(const ssd_selective_shape* shape) {
  SelDims d;
  if (sel_dims(shape, &d) != SSD_OK || bwd_chunks(&d) != SSD_OK) return 0;
  return bwd_ws(d, nullptr).total;
}

int ssd_selective_scan_fwd(const ssd_selective_shape* shape, const void* x, const void* dt,
                           const float* dt_bias, const float* A, const void* B, const void* C,
                           const float* D, const void* z, const float* init_states,
                           const int32_t* lengths, void* out, float* final_states,
                           void* workspace, size_t workspace_bytes, void* stream) {
  SelDims d;
  int st = sel_dims(shape, &d);
  if (st == SSD_OK) st = fwd_chunks(&d);
  if (st != SSD_OK) return st;
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4, oe = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (!x || !dt || !A || !B || !C || !out) return SSD_ERR_INVALID_ARG;
  if (off(x, ie) || off(dt, ie) || off(B, ie) || off(C, ie) || off(z, ie) || off(out, oe) ||
      off(dt_bias, 4) || off(A, 4) || off(D, 4) || off(init_states, 4) || off(final_states, 4) ||
      off(lengths, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || off(workspace, 16) ||
      workspace_bytes < ssd_selective_scan_fwd_workspace_size(shape))
    return SSD_ERR_WORKSPACE;
  float* hin = static_cast<float*>(workspace);
  float* sumd = reinterpret_cast<float*>(
      static_cast<char*>(workspace) +
      align_up((size_t)d.B * d.nc * d.D * d.N * sizeof(float), 256));
  const SelIn in{x, dt, dt_bias, A, B, C, D, z, lengths};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* const ins[3] = {x, dt, nullptr};
  const void* const outs[3] = {out, nullptr, nullptr};
  const void* const states[3] = {A, init_states, final_states};
  access(&d, ie, oe, ins, outs, z, states);
  return by_states(d.N, [&](auto spt, auto sl) {
#define SSD_GO(TI, TO, ODD)                                                                   \
  sel_forward<TI, TO, spt(), sl(), ODD>(d, in, init_states, out, final_states, hin, sumd, s)
    if (ie == 4) return SSD_GO(float, float, false);
    if (d.mode == 1) return oe == 4 ? SSD_GO(bf16, float, true) : SSD_GO(bf16, bf16, true);
    return oe == 4 ? SSD_GO(bf16, float, false) : SSD_GO(bf16, bf16, false);
#undef SSD_GO
  });
}

int ssd_selective_scan_bwd(const ssd_selective_shape* shape, const void* x, const void* dt,
                           const float* dt_bias, const float* A, const void* B, const void* C,
                           const float* D, const void* z, const float* init_states,
                           const int32_t* lengths, const void* dout, const float* dfinal_states,
                           void* dx, void* ddt, float* dA, float* dB, float* dC, float* dD,
                           void* dz, float* ddt_bias, float* dinit_states, void* workspace,
                           size_t workspace_bytes, void* stream) {
  SelDims d;
  int st = sel_dims(shape, &d);
  if (st == SSD_OK) st = bwd_chunks(&d);
  if (st != SSD_OK) return st;
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4, oe = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (!x || !dt || !A || !B || !C || !dout || !dx || !ddt || !dA || !dB || !dC || (z && !dz))
    return SSD_ERR_INVALID_ARG;
  if (off(x, ie) || off(dt, ie) || off(B, ie) || off(C, ie) || off(z, ie) || off(dout, ie) ||
      off(dx, oe) || off(ddt, oe) || off(dz, oe) || off(dt_bias, 4) || off(A, 4) || off(D, 4) ||
      off(init_states, 4) || off(lengths, 4) || off(dfinal_states, 4) || off(dA, 4) ||
      off(dB, 4) || off(dC, 4) || off(dD, 4) || off(ddt_bias, 4) || off(dinit_states, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || off(workspace, 16) ||
      workspace_bytes < ssd_selective_scan_bwd_workspace_size(shape))
    return SSD_ERR_WORKSPACE;
  const SelBwdWs w = bwd_ws(d, workspace);
  const SelIn in{x, dt, dt_bias, A, B, C, D, z, lengths};
  const SelGrads g{dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit_states};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* const ins[3] = {x, dt, dout};
  const void* const outs[3] = {dz, nullptr, nullptr};
  const void* const states[3] = {A, dinit_states, nullptr};
  access(&d, ie, oe, ins, outs, z, states);
  return by_states(d.N, [&](auto spt, auto sl) {
#define SSD_GO(TI, TO, ODD)                                                                   \
  sel_backward<TI, TO, spt(), sl(), ODD>(d, in, init_states, dout, dfinal_states, g, w, s)
    if (ie == 4) return SSD_GO(float, float, false);
    if (d.mode == 1) return oe == 4 ? SSD_GO(bf16, float, true) : SSD_GO(bf16, bf16, true);
    return oe == 4 ? SSD_GO(bf16, float, false) : SSD_GO(bf16, bf16, false);
#undef SSD_GO
  });
}

}  // extern "C"
