// Selective scan with a decay per channel and state (the first-generation
// Mamba recurrence): for batch b, channel d of group g(d) and state n
//     delta = softplus(dt + dt_bias)
//     h[n]  = exp(delta A[d, n]) h[n] + delta x B[n]
//     y     = sum_n C[n] h[n] + D[d] x,   out = y silu(z)  (or y without z)
// and its backward.  The pages' scan has one scalar decay per head, which
// turns a chunk into matrix products; with a decay per (d, n) there is no such
// product, and every (position, channel, state) costs one exponential and four
// operations of the FMA pipe: the arithmetic binds, not HBM.
//
// The sequence is cut into chunks that run in parallel, since B x channels
// alone leaves most of the machine idle:
//     k_sel_state    each chunk's state from zero, and the sum of its deltas
//     k_sel_combine  the state entering each chunk (decays exp(A sum delta))
//     k_sel_scan     each chunk again from its state, with the outputs
// and in the backward
//     k_sel_state    also each chunk's adjoint at its start, from zero after it:
//                    sum_t exp(A (delta_1 + .. + delta_t)) C_t dy_t
//     k_sel_combine  also the adjoint entering each chunk from the right
//     k_sel_bwd      the gradients of a chunk
//     k_sel_bc, k_sel_params  fixed-order sums of dB, dC and of dA, dD, ddt_bias
// A warp owns CL = 32 / SL channel lanes (times CPT channels each) and SL
// state lanes of SPT states each, all in registers; the sum over the states of
// an output is mostly lane-local.
#include <cuda_bf16.h>

#include "layer_math.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace lm;
using bf16 = __nv_bfloat16;

struct SelDims {
  int B, T, D, N, G, DG;  // DG: channels per group
  int L, nc;              // chunk length and count
  int ctiles;             // blocks' channel tiles per group
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

// A block's place: batch row, group, chunk and first channel of the group.
struct Place {
  int b, g, c, q0;
};
__device__ __forceinline__ Place place(const SelDims& d, int channels) {
  Place p;
  int i = blockIdx.x;
  const int ct = i % d.ctiles;
  i /= d.ctiles;
  p.g = i % d.G;
  p.b = i / d.G;
  p.c = blockIdx.y;
  p.q0 = ct * channels;
  return p;
}

// Rows [t0, t0 + nt) of B (and C) of one group as fp32 in shared memory,
// padded with zeros to NP states and past position n.
template <typename Tin, int NP>
__device__ __forceinline__ void stage_rows(float* dst, const Tin* src, int64_t stride, int N,
                                           int t0, int nt, int n) {
  for (int i = threadIdx.x; i < nt * NP; i += blockDim.x) {
    const int t = i / NP, k = i - t * NP;
    dst[i] = (k < N && t0 + t < n) ? to_f(src[(int64_t)(t0 + t) * stride + k]) : 0.f;
  }
}

constexpr int kTile = 32;  // positions of B and C staged at a time

// Sum over the state lanes (lane = sl * CL + cl).
template <int SL>
__device__ __forceinline__ float sum_states(float v) {
#pragma unroll
  for (int o = 32 / SL; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kFwdWarps = 4;

// Forward pass over one chunk.  OUT: with the outputs, from the state
// hin (B, nc, D, N) (or init when there is one chunk); else the chunk's state
// from zero into hin and its delta sum into sumd (B, nc, D).
template <typename Tin, typename Tout, int SPT, int SL, int CPT, bool OUT>
__global__ void __launch_bounds__(32 * kFwdWarps)
    k_sel_scan(SelIn in, const float* __restrict__ init, float* __restrict__ hin,
               float* __restrict__ sumd, Tout* __restrict__ out, float* __restrict__ final_state,
               SelDims d) {
  constexpr int CL = 32 / SL, NP = SPT * SL, CW = CL * CPT;
  __shared__ __align__(16) float sB[kTile * NP], sC[OUT ? kTile * NP : 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sl = lane / CL, cl = lane % CL;
  const Place p = place(d, CW * kFwdWarps);
  const int n = sel_len(in.lengths, p.b, d.T);
  const int64_t row0 = (int64_t)p.b * d.T;
  const Tin* x = static_cast<const Tin*>(in.x) + row0 * d.D;
  const Tin* dt = static_cast<const Tin*>(in.dt) + row0 * d.D;
  const Tin* z = in.z ? static_cast<const Tin*>(in.z) + p.b * d.zb : nullptr;
  const Tin* Bm = static_cast<const Tin*>(in.B) + p.b * d.bb + (int64_t)p.g * d.N;
  const Tin* Cm = static_cast<const Tin*>(in.C) + p.b * d.cb + (int64_t)p.g * d.N;

  int ch[CPT];
  bool on[CPT];
  float a2[CPT][SPT], h[CPT][SPT], bias[CPT], skip[CPT], sd[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int q = p.q0 + warp * CW + j * CL + cl;
    on[j] = q < d.DG;
    ch[j] = p.g * d.DG + (on[j] ? q : 0);
    bias[j] = in.dt_bias && on[j] ? in.dt_bias[ch[j]] : 0.f;
    skip[j] = in.D && on[j] ? in.D[ch[j]] : 0.f;
    sd[j] = 0.f;
    const float* h0 = nullptr;
    if (OUT && on[j]) {
      if (d.nc > 1)
        h0 = hin + (((int64_t)p.b * d.nc + p.c) * d.D + ch[j]) * d.N;
      else if (init)
        h0 = init + ((int64_t)p.b * d.D + ch[j]) * d.N;
    }
#pragma unroll
    for (int k = 0; k < SPT; ++k) {
      const int s = sl * SPT + k;
      a2[j][k] = on[j] && s < d.N ? in.A[(int64_t)ch[j] * d.N + s] * kLog2e : 0.f;
      h[j][k] = h0 && s < d.N ? h0[s] : 0.f;
    }
  }
  const int t0 = p.c * d.L, t1 = min(d.T, t0 + d.L), tv = min(t1, n);
  for (int tb = t0; tb < tv; tb += kTile) {
    __syncthreads();
    stage_rows<Tin, NP>(sB, Bm, d.bs, d.N, tb, kTile, tv);
    if (OUT) stage_rows<Tin, NP>(sC, Cm, d.cs, d.N, tb, kTile, tv);
    __syncthreads();
    const int te = min(kTile, tv - tb);
    for (int t = 0; t < te; ++t) {
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int64_t at = (int64_t)(tb + t) * d.D + ch[j];
        const float xv = to_f(x[at]);
        const float delta = softplus(to_f(dt[at]) + bias[j]);
        const float dtx = delta * xv;
        sd[j] += delta;
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < SPT; ++k) {
          h[j][k] = fmaf(ex2(delta * a2[j][k]), h[j][k], dtx * sB[t * NP + sl * SPT + k]);
          if (OUT) y = fmaf(h[j][k], sC[t * NP + sl * SPT + k], y);
        }
        if (OUT) {
          y = sum_states<SL>(y);
          if (sl == 0 && on[j]) {
            y = fmaf(skip[j], xv, y);
            if (z) {
              const float zv = to_f(z[(int64_t)(tb + t) * d.zs + ch[j]]);
              y *= zv * sigmoid(zv);
            }
            out[row0 * d.D + at] = from_f<Tout>(y);
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (!on[j]) continue;
    if (OUT) {
      if (sl == 0)
        for (int t = max(t0, tv); t < t1; ++t)
          out[(row0 + t) * d.D + ch[j]] = from_f<Tout>(0.f);
      if (final_state && p.c == d.nc - 1)
#pragma unroll
        for (int k = 0; k < SPT; ++k)
          if (sl * SPT + k < d.N)
            final_state[((int64_t)p.b * d.D + ch[j]) * d.N + sl * SPT + k] = h[j][k];
    } else {
      const int64_t at = ((int64_t)p.b * d.nc + p.c) * d.D + ch[j];
      if (sl == 0) sumd[at] = sd[j];
#pragma unroll
      for (int k = 0; k < SPT; ++k)
        if (sl * SPT + k < d.N) hin[at * d.N + sl * SPT + k] = h[j][k];
    }
  }
}

// The backward's first pass: each chunk's state from zero (hin), its delta
// sum and its adjoint at its start from zero after it (gin).  Running products
// of the decays give the adjoint in the forward direction, from the same
// exponentials.
template <typename Tin, int SPT, int SL>
__global__ void __launch_bounds__(32 * kFwdWarps)
    k_sel_state(SelIn in, const Tin* __restrict__ dout, float* __restrict__ hin,
                float* __restrict__ gin, float* __restrict__ sumd, SelDims d) {
  constexpr int CL = 32 / SL, NP = SPT * SL, CW = CL;
  __shared__ __align__(16) float sB[kTile * NP], sC[kTile * NP];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sl = lane / CL, cl = lane % CL;
  const Place p = place(d, CW * kFwdWarps);
  const int n = sel_len(in.lengths, p.b, d.T);
  const int64_t row0 = (int64_t)p.b * d.T;
  const Tin* x = static_cast<const Tin*>(in.x) + row0 * d.D;
  const Tin* dt = static_cast<const Tin*>(in.dt) + row0 * d.D;
  const Tin* z = in.z ? static_cast<const Tin*>(in.z) + p.b * d.zb : nullptr;
  const Tin* Bm = static_cast<const Tin*>(in.B) + p.b * d.bb + (int64_t)p.g * d.N;
  const Tin* Cm = static_cast<const Tin*>(in.C) + p.b * d.cb + (int64_t)p.g * d.N;
  dout += row0 * d.D;
  const int q = p.q0 + warp * CW + cl;
  const bool on = q < d.DG;
  const int ch = p.g * d.DG + (on ? q : 0);
  const float bias = in.dt_bias && on ? in.dt_bias[ch] : 0.f;
  float a2[SPT], h[SPT], pr[SPT], gl[SPT], sd = 0.f;
#pragma unroll
  for (int k = 0; k < SPT; ++k) {
    const int s = sl * SPT + k;
    a2[k] = on && s < d.N ? in.A[(int64_t)ch * d.N + s] * kLog2e : 0.f;
    h[k] = gl[k] = 0.f;
    pr[k] = 1.f;
  }
  const int t0 = p.c * d.L, t1 = min(d.T, t0 + d.L), tv = min(t1, n);
  for (int tb = t0; tb < tv; tb += kTile) {
    __syncthreads();
    stage_rows<Tin, NP>(sB, Bm, d.bs, d.N, tb, kTile, tv);
    stage_rows<Tin, NP>(sC, Cm, d.cs, d.N, tb, kTile, tv);
    __syncthreads();
    const int te = min(kTile, tv - tb);
    for (int t = 0; t < te; ++t) {
      const int64_t at = (int64_t)(tb + t) * d.D + ch;
      const float delta = softplus(to_f(dt[at]) + bias);
      const float dtx = delta * to_f(x[at]);
      float dy = to_f(dout[at]);
      if (z) {
        const float zv = to_f(z[(int64_t)(tb + t) * d.zs + ch]);
        dy *= zv * sigmoid(zv);
      }
      sd += delta;
#pragma unroll
      for (int k = 0; k < SPT; ++k) {
        const float a = ex2(delta * a2[k]);
        h[k] = fmaf(a, h[k], dtx * sB[t * NP + sl * SPT + k]);
        pr[k] *= a;
        gl[k] = fmaf(pr[k], dy * sC[t * NP + sl * SPT + k], gl[k]);
      }
    }
  }
  if (!on) return;
  const int64_t at = ((int64_t)p.b * d.nc + p.c) * d.D + ch;
  if (sl == 0) sumd[at] = sd;
#pragma unroll
  for (int k = 0; k < SPT; ++k)
    if (sl * SPT + k < d.N) {
      hin[at * d.N + sl * SPT + k] = h[k];
      gin[at * d.N + sl * SPT + k] = gl[k];
    }
}

// hin: each chunk's own state -> the state entering it, in place:
// H_{c+1} = exp(A sumd_c) H_c + S_c.  With gin (blockIdx.y = 1): each chunk's own
// adjoint at its start -> the adjoint entering it from the right:
// G_c = gin_c + exp(A sumd_c) G_{c+1}.  One thread per (b, d, n).
__global__ void __launch_bounds__(256)
    k_sel_combine(const float* __restrict__ A, const float* __restrict__ init,
                  const float* __restrict__ dfinal, float* __restrict__ hin,
                  float* __restrict__ gin, const float* __restrict__ sumd, SelDims d) {
  const int64_t DN = (int64_t)d.D * d.N, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= d.B * DN) return;
  const int b = (int)(i / DN);
  const int64_t dn = i - b * DN;
  const int ch = (int)(dn / d.N);
  const float a2 = A[dn] * kLog2e;
  const bool rev = blockIdx.y == 1;
  float* v = (rev ? gin : hin) + (int64_t)b * d.nc * DN + dn;
  const float* sm = sumd + (int64_t)b * d.nc * d.D + ch;
  const float* start = rev ? dfinal : init;
  float acc = start ? start[i] : 0.f;
  constexpr int U = 4;
  for (int c0 = 0; c0 < d.nc; c0 += U) {
    float e[U], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = rev ? d.nc - 1 - c0 - u : c0 + u;
      const bool in = c0 + u < d.nc;
      // the last chunk's own state is not needed (the forward writes none)
      s[u] = in && c0 + u < d.nc - 1 ? v[c * DN] : 0.f;
      e[u] = in ? sm[(int64_t)c * d.D] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = rev ? d.nc - 1 - c0 - u : c0 + u;
      if (c0 + u < d.nc) {
        v[c * DN] = acc;
        acc = fmaf(ex2(e[u] * a2), acc, s[u]);
      }
    }
  }
}

// Sums v[0 .. NV) over the CL lanes cl of a state lane.  Halving exchanges: at
// each step a lane keeps one half of the values and sends the other to the
// lane that keeps that one, so lane cl ends with the totals
// [cl * NV / CL, (cl + 1) * NV / CL) in v[0 ..]; with fewer values than lanes,
// CL / NV consecutive lanes end with the total cl / (CL / NV).
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

constexpr int kBwdL = 32, kBwdTS = 4, kBwdWarps = 4;
constexpr int kBwdTiles = kBwdL / kBwdTS;

template <int SPT, int SL>
struct BwdSmem {
  static constexpr int NP = SPT * SL, CW = 32 / SL;
  float B[kBwdL * NP], C[kBwdL * NP];
  float red[kBwdWarps][kBwdTS][2 * NP];
  float delta[kBwdWarps][kBwdL][CW], dy[kBwdWarps][kBwdL][CW], x[kBwdWarps][kBwdL][CW];
  float start[kBwdWarps][kBwdTiles][SPT][32];
};

// Gradients of one chunk of kBwdL positions.  With the state and the adjoint
// that enter it known, the warp walks forward once, keeping the state at every
// kBwdTS-th position, then backward tile by tile: the tile's states are formed
// again into registers, and at each position
//     g = C dy + a_next g_next,  w = (a g) h_prev
//     dA += delta w,  ddelta = sum_n (A w + x g B),  dx = delta sum_n g B + D dy
//     dB_t += delta x g,  dC_t += dy h   (sums over the group's channels).
// The last two are sums over lanes: halving exchanges leave each lane one
// total (31 shuffles for 32 values), the block's warps are added in shared
// memory, and each block writes its part (B, T, G, ctiles, 2 N).
template <typename Tin, typename Tout, int SPT, int SL>
__global__ void __launch_bounds__(32 * kBwdWarps)
    k_sel_bwd(SelIn in, const Tin* __restrict__ dout, const float* __restrict__ hin,
              const float* __restrict__ gin, Tout* __restrict__ dx, Tout* __restrict__ ddt,
              Tout* __restrict__ dz, float* __restrict__ bcpart, float* __restrict__ dApart,
              float* __restrict__ ppart, float* __restrict__ dinit, SelDims d) {
  constexpr int CL = 32 / SL, NP = SPT * SL, CW = CL, NV = 2 * SPT;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  BwdSmem<SPT, SL>& sm = *reinterpret_cast<BwdSmem<SPT, SL>*>(raw_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sl = lane / CL, cl = lane % CL;
  const Place p = place(d, CW * kBwdWarps);
  const int n = sel_len(in.lengths, p.b, d.T);
  const int64_t row0 = (int64_t)p.b * d.T;
  const Tin* x = static_cast<const Tin*>(in.x) + row0 * d.D;
  const Tin* dt = static_cast<const Tin*>(in.dt) + row0 * d.D;
  const Tin* z = in.z ? static_cast<const Tin*>(in.z) + p.b * d.zb : nullptr;
  const Tin* Bm = static_cast<const Tin*>(in.B) + p.b * d.bb + (int64_t)p.g * d.N;
  const Tin* Cm = static_cast<const Tin*>(in.C) + p.b * d.cb + (int64_t)p.g * d.N;
  dout += row0 * d.D;
  const int t0 = p.c * kBwdL, t1 = min(d.T, t0 + kBwdL), tv = min(t1, n);
  const int qw = p.q0 + warp * CW, q = qw + cl;
  const bool on = q < d.DG;
  const int ch = p.g * d.DG + (on ? q : 0);
  const float bias = in.dt_bias && on ? in.dt_bias[ch] : 0.f;

  // one lane in SL computes a (position, channel)'s delta, x and dy
  stage_rows<Tin, NP>(sm.B, Bm, d.bs, d.N, t0, kBwdL, tv);
  stage_rows<Tin, NP>(sm.C, Cm, d.cs, d.N, t0, kBwdL, tv);
  for (int t = sl; t < kBwdL; t += SL) {
    float dl = 0.f, xv = 0.f, dy = 0.f;
    if (on && t0 + t < tv) {
      const int64_t at = (int64_t)(t0 + t) * d.D + ch;
      xv = to_f(x[at]);
      dl = softplus(to_f(dt[at]) + bias);
      dy = to_f(dout[at]);
      if (z) {
        const float zv = to_f(z[(int64_t)(t0 + t) * d.zs + ch]);
        dy *= zv * sigmoid(zv);
      }
    }
    sm.delta[warp][t][cl] = dl;
    sm.x[warp][t][cl] = xv;
    sm.dy[warp][t][cl] = dy;
  }
  __syncthreads();

  float a2[SPT], h[SPT], gc[SPT], dA[SPT];
  const int64_t cat = ((int64_t)p.b * d.nc + p.c) * d.D + ch;
#pragma unroll
  for (int k = 0; k < SPT; ++k) {
    const int s = sl * SPT + k;
    const bool ok = on && s < d.N;
    a2[k] = ok ? in.A[(int64_t)ch * d.N + s] * kLog2e : 0.f;
    h[k] = ok ? hin[cat * d.N + s] : 0.f;
    gc[k] = ok ? gin[cat * d.N + s] : 0.f;
    dA[k] = 0.f;
  }
  for (int t = 0; t < kBwdL; ++t) {
    if (t % kBwdTS == 0) {
#pragma unroll
      for (int k = 0; k < SPT; ++k) sm.start[warp][t / kBwdTS][k][lane] = h[k];
      if (t == kBwdL - kBwdTS) break;
    }
    const float dl = sm.delta[warp][t][cl], dtx = dl * sm.x[warp][t][cl];
#pragma unroll
    for (int k = 0; k < SPT; ++k)
      h[k] = fmaf(ex2(dl * a2[k]), h[k], dtx * sm.B[t * NP + sl * SPT + k]);
  }
  const float skip = in.D && on ? in.D[ch] : 0.f;
  float dD = 0.f, dbias = 0.f;
  for (int tile = kBwdTiles - 1; tile >= 0; --tile) {
    float hs[kBwdTS][SPT];
#pragma unroll
    for (int k = 0; k < SPT; ++k) h[k] = sm.start[warp][tile][k][lane];
#pragma unroll
    for (int u = 0; u < kBwdTS; ++u) {
      const int t = tile * kBwdTS + u;
      const float dl = sm.delta[warp][t][cl], dtx = dl * sm.x[warp][t][cl];
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < SPT; ++k) {
        h[k] = fmaf(ex2(dl * a2[k]), h[k], dtx * sm.B[t * NP + sl * SPT + k]);
        hs[u][k] = h[k];
        y = fmaf(h[k], sm.C[t * NP + sl * SPT + k], y);
      }
      if (z) {
        y = sum_states<SL>(y);
        if (sl == u % SL && on && t0 + t < t1) {
          float o = 0.f;
          if (t0 + t < tv) {
            const float zv = to_f(z[(int64_t)(t0 + t) * d.zs + ch]), sg = sigmoid(zv);
            y = fmaf(skip, sm.x[warp][t][cl], y);
            o = to_f(dout[(int64_t)(t0 + t) * d.D + ch]) * y * sg * (1.f + zv * (1.f - sg));
          }
          dz[(row0 + t0 + t) * d.D + ch] = from_f<Tout>(o);
        }
      }
    }
#pragma unroll
    for (int u = kBwdTS - 1; u >= 0; --u) {
      const int t = tile * kBwdTS + u;
      const float dl = sm.delta[warp][t][cl], xv = sm.x[warp][t][cl], dy = sm.dy[warp][t][cl];
      const float dtx = dl * xv;
      float v[NV], gb = 0.f, aw = 0.f;
#pragma unroll
      for (int k = 0; k < SPT; ++k) {
        const float Bk = sm.B[t * NP + sl * SPT + k], Ck = sm.C[t * NP + sl * SPT + k];
        const float g = fmaf(Ck, dy, gc[k]);
        gc[k] = ex2(dl * a2[k]) * g;
        const float w = gc[k] * (u > 0 ? hs[u > 0 ? u - 1 : 0][k] : sm.start[warp][tile][k][lane]);
        dA[k] = fmaf(dl, w, dA[k]);
        aw = fmaf(a2[k], w, aw);
        gb = fmaf(g, Bk, gb);
        v[k] = dtx * g;
        v[SPT + k] = dy * hs[u][k];
      }
      reduce_lanes<NV, CL>(v, cl);
      constexpr int kPer = NV > CL ? NV / CL : 1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int idx = cl * NV / CL + i;  // < SPT: dB, else dC, of this state lane
        sm.red[warp][u][(idx / SPT) * NP + sl * SPT + idx % SPT] = v[i];
      }
      gb = sum_states<SL>(gb);
      aw = sum_states<SL>(aw) * 0.6931471805599453f;  // a2 = A log2(e)
      if (sl == u % SL && on && t0 + t < t1) {
        const int64_t at = (int64_t)(t0 + t) * d.D + ch;
        float dv = 0.f;
        if (t0 + t < tv) dv = fmaf(xv, gb, aw) * sigmoid(to_f(dt[at]) + bias);
        dx[row0 * d.D + at] = from_f<Tout>(fmaf(dl, gb, skip * dy));
        ddt[row0 * d.D + at] = from_f<Tout>(dv);
        dD = fmaf(dy, xv, dD);
        dbias += dv;
      }
    }
    __syncthreads();
    const int ct = p.q0 / (CW * kBwdWarps);
    for (int i = threadIdx.x; i < kBwdTS * 2 * NP; i += blockDim.x) {
      const int u = i / (2 * NP), e = i - u * (2 * NP), s = e % NP, t = t0 + tile * kBwdTS + u;
      if (s < d.N && t < t1) {
        float a = 0.f;
#pragma unroll
        for (int wv = 0; wv < kBwdWarps; ++wv) a += sm.red[wv][u][e];
        bcpart[(((row0 + t) * d.G + p.g) * d.ctiles + ct) * (2 * d.N) + (e / NP) * d.N + s] = a;
      }
    }
    __syncthreads();
  }
  dD = sum_states<SL>(dD);
  dbias = sum_states<SL>(dbias);
  if (!on) return;
  if (sl == 0) {
    ppart[cat * 2] = dD;
    ppart[cat * 2 + 1] = dbias;
  }
#pragma unroll
  for (int k = 0; k < SPT; ++k) {
    const int s = sl * SPT + k;
    if (s < d.N) {
      dApart[cat * d.N + s] = dA[k];
      if (dinit && p.c == 0) dinit[((int64_t)p.b * d.D + ch) * d.N + s] = gc[k];
    }
  }
}

// dB, dC (B, T, G, N): the channel tiles' parts, in order.
__global__ void __launch_bounds__(256)
    k_sel_bc(const float* __restrict__ part, float* __restrict__ dB, float* __restrict__ dC,
             int64_t rows, int ctiles, int N) {
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

int state_lanes(int N) { return N > 32 ? 4 : N > 16 ? 2 : 1; }
constexpr int kCPT = 2;

// Forward chunks: as many as give about 12 warps per SM, at least two
// staged tiles long; one chunk (no state pass) where the channels fill half of
// that by themselves.
void fwd_chunks(SelDims* d) {
  const int chans = 32 / state_lanes(d->N) * kCPT * kFwdWarps;
  d->ctiles = ceil_div(d->DG, chans);
  const int64_t blocks = (int64_t)d->B * d->G * d->ctiles;
  int64_t nc = 3 * 152 / blocks;
  const int64_t most = ceil_div(d->T, 2 * kTile);
  if (nc > most) nc = most;
  if (nc < 2) nc = 1;
  d->L = ceil_div(ceil_div(d->T, nc), kTile) * kTile;
  d->nc = ceil_div(d->T, d->L);
}

void bwd_chunks(SelDims* d) {
  d->ctiles = ceil_div(d->DG, 32 / state_lanes(d->N) * kBwdWarps);
  d->L = kBwdL;
  d->nc = ceil_div(d->T, kBwdL);
}

struct SelBwdWs {
  float *hin, *gin, *sumd, *bc, *dA, *pp;
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
  const size_t cd = (size_t)d.B * d.nc * d.D;
  w.hin = take(cd * d.N);
  w.gin = take(cd * d.N);
  w.sumd = take(cd);
  w.dA = take(cd * d.N);
  w.pp = take(cd * 2);
  w.bc = take((size_t)d.B * d.T * d.G * d.ctiles * 2 * d.N);
  w.total = off;
  return w;
}

dim3 sel_grid(const SelDims& d, int chunks) {
  return dim3((unsigned)((int64_t)d.B * d.G * d.ctiles), chunks);
}

cudaError_t combine(const SelDims& d, const float* A, const float* init, const float* dfinal,
                    float* hin, float* gin, const float* sumd, cudaStream_t s) {
  const int64_t n = (int64_t)d.B * d.D * d.N;
  const dim3 grid((unsigned)((n + 255) / 256), gin ? 2 : 1);
  SSD_LAUNCH("k_sel_combine", s,
             k_sel_combine<<<grid, 256, 0, s>>>(A, init, dfinal, hin, gin, sumd, d));
  return cudaGetLastError();
}

template <typename Tin, typename Tout, int SPT, int SL>
int sel_forward(const SelDims& d, const SelIn& in, const float* init, void* out, float* fin,
                float* hin, float* sumd, cudaStream_t s) {
  if (d.nc > 1) {
    SSD_LAUNCH("k_sel_chunk_state", s,
               k_sel_scan<Tin, Tout, SPT, SL, kCPT, false>
               <<<sel_grid(d, d.nc - 1), 32 * kFwdWarps, 0, s>>>(in, nullptr, hin, sumd, nullptr,
                                                                 nullptr, d));
    if (combine(d, in.A, init, nullptr, hin, nullptr, sumd, s) != cudaSuccess) return SSD_ERR_CUDA;
  }
  SSD_LAUNCH("k_sel_scan", s,
             k_sel_scan<Tin, Tout, SPT, SL, kCPT, true>
             <<<sel_grid(d, d.nc), 32 * kFwdWarps, 0, s>>>(in, init, hin, nullptr,
                                                           static_cast<Tout*>(out), fin, d));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

struct SelGrads {
  void *dx, *ddt;
  float *dA, *dB, *dC, *dD;
  void* dz;
  float *ddt_bias, *dinit;
};

template <typename Tin, typename Tout, int SPT, int SL>
int sel_backward(const SelDims& d, const SelIn& in, const float* init, const void* dout,
                 const float* dfinal, const SelGrads& g, const SelBwdWs& w, cudaStream_t s) {
  const Tin* go = static_cast<const Tin*>(dout);
  SSD_LAUNCH("k_sel_state", s,
             k_sel_state<Tin, SPT, SL><<<sel_grid(d, d.nc), 32 * kFwdWarps, 0, s>>>(
                 in, go, w.hin, w.gin, w.sumd, d));
  if (combine(d, in.A, init, dfinal, w.hin, w.gin, w.sumd, s) != cudaSuccess) return SSD_ERR_CUDA;
  auto kern = k_sel_bwd<Tin, Tout, SPT, SL>;
  constexpr size_t smem = sizeof(BwdSmem<SPT, SL>);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return SSD_ERR_CUDA;
  SSD_LAUNCH("k_sel_bwd", s,
             kern<<<sel_grid(d, d.nc), 32 * kBwdWarps, smem, s>>>(
                 in, go, w.hin, w.gin, static_cast<Tout*>(g.dx), static_cast<Tout*>(g.ddt),
                 static_cast<Tout*>(g.dz), w.bc, w.dA, w.pp, g.dinit, d));
  const int64_t rows = (int64_t)d.B * d.T * d.G, DN = (int64_t)d.D * d.N;
  SSD_LAUNCH("k_sel_bc", s,
             k_sel_bc<<<(unsigned)((rows * 2 * d.N + 255) / 256), 256, 0, s>>>(
                 w.bc, g.dB, g.dC, rows, d.ctiles, d.N));
  const int ba = ceil_div(DN, 32), bp = ceil_div(2 * (int64_t)d.D, 32);
  SSD_LAUNCH("k_sel_params", s,
             k_sel_params<<<ba + bp, 256, 0, s>>>(w.dA, w.pp, g.dA, g.dD, g.ddt_bias, d.B * d.nc,
                                                  DN, d.D, ba));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// The instantiation for a state count and a pair of types.
template <typename F>
int by_states(int N, F&& f) {
  if (N <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (N <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (N <= 32) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
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
  if (sel_dims(shape, &d) != SSD_OK) return 0;
  fwd_chunks(&d);
  if (d.nc == 1) return 256;
  const size_t cd = (size_t)d.B * d.nc * d.D;
  return align_up(cd * d.N * sizeof(float), 256) + align_up(cd * sizeof(float), 256);
}

size_t ssd_selective_scan_bwd_workspace_size(const ssd_selective_shape* shape) {
  SelDims d;
  if (sel_dims(shape, &d) != SSD_OK) return 0;
  bwd_chunks(&d);
  return bwd_ws(d, nullptr).total;
}

int ssd_selective_scan_fwd(const ssd_selective_shape* shape, const void* x, const void* dt,
                           const float* dt_bias, const float* A, const void* B, const void* C,
                           const float* D, const void* z, const float* init_states,
                           const int32_t* lengths, void* out, float* final_states,
                           void* workspace, size_t workspace_bytes, void* stream) {
  SelDims d;
  const int st = sel_dims(shape, &d);
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
  fwd_chunks(&d);
  if ((int64_t)d.B * d.G * d.ctiles > 0x7fffffff || d.nc > 65535) return SSD_ERR_UNSUPPORTED;
  float* hin = static_cast<float*>(workspace);
  float* sumd = reinterpret_cast<float*>(
      static_cast<char*>(workspace) +
      align_up((size_t)d.B * d.nc * d.D * d.N * sizeof(float), 256));
  const SelIn in{x, dt, dt_bias, A, B, C, D, z, lengths};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_states(d.N, [&](auto spt, auto sl) {
    if (ie == 4)
      return sel_forward<float, float, spt(), sl()>(d, in, init_states, out, final_states, hin, sumd, s);
    if (oe == 4)
      return sel_forward<bf16, float, spt(), sl()>(d, in, init_states, out, final_states, hin, sumd, s);
    return sel_forward<bf16, bf16, spt(), sl()>(d, in, init_states, out, final_states, hin, sumd, s);
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
  const int st = sel_dims(shape, &d);
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
  bwd_chunks(&d);
  if ((int64_t)d.B * d.G * d.ctiles > 0x7fffffff || d.nc > 65535) return SSD_ERR_UNSUPPORTED;
  const SelBwdWs w = bwd_ws(d, workspace);
  const SelIn in{x, dt, dt_bias, A, B, C, D, z, lengths};
  const SelGrads g{dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit_states};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_states(d.N, [&](auto spt, auto sl) {
    if (ie == 4)
      return sel_backward<float, float, spt(), sl()>(d, in, init_states, dout, dfinal_states, g, w, s);
    if (oe == 4)
      return sel_backward<bf16, float, spt(), sl()>(d, in, init_states, dout, dfinal_states, g, w, s);
    return sel_backward<bf16, bf16, spt(), sl()>(d, in, init_states, dout, dfinal_states, g, w, s);
  });
}

}  // extern "C"
