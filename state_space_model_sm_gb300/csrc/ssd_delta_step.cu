// One token of the gated delta rule, for decoding: with a = exp(softplus(dt +
// dt_bias) A) and b = sigmoid(beta),
//     u = b (v - a S k),   S <- a S + u k^T,   y = scale S q
// for every value row of a head's state, in a cache of slots.
//
// The state is read and written once, 8 bytes for 8 operations: HBM-bound.  A row's
// dstate values lie across the LPR lanes of a warp segment, V at a time and NV times,
// and stay in registers between the two passes over them; each lane holds RB rows, and
// they are the first thing loaded, so that the latency of the gates lies under theirs.
// Both dots of a row come from the state as it was read: S k, and S q with
//     y = scale (a S q + u (k . q)),
// so a row is summed over the lanes once.
//
// 128 rows of 32 heads of 128 x 128 take 84 us, 6.4 TB/s: 95 % of the measured copy rate.
// One row of 24 heads of 64 x 128 takes 2.4 us in a row of launches, which is a launch.
#include <cuda_bf16.h>

#include "layer_math.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace lm;
using bf16 = __nv_bfloat16;

struct DeltaStepDims {
  int B, H, G, P, N;
  int RG;     // state rows of a group
  int tiles;  // warp tiles of a group
  int64_t qs, ks, vs;
  float scale;
};

constexpr int kStepWarps = 4;

template <typename Tin, typename Tout, int LPR, int V, int NV, int RB>
__global__ void __launch_bounds__(32 * kStepWarps)
    k_delta_step(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
                 const Tin* __restrict__ dt, const float* __restrict__ dt_bias,
                 const float* __restrict__ A, const Tin* __restrict__ beta, float* __restrict__ state,
                 const int* __restrict__ slots, int64_t nslots, Tout* __restrict__ y,
                 DeltaStepDims d) {
  constexpr int RPW = 32 / LPR;  // rows of a warp at a time
  static_assert(RB <= LPR, "each of a segment's RB rows has a lane of its own");
  const int lane = threadIdx.x & 31, seg = lane / LPR, sl = lane % LPR;
  const int64_t tile = (int64_t)blockIdx.x * kStepWarps + (threadIdx.x >> 5);
  const int64_t bg = tile / d.tiles;
  const int b = (int)(bg / d.G), g = (int)(bg - (int64_t)b * d.G);
  if (b >= d.B) return;
  const int q0 = (int)(tile - bg * d.tiles) * (RB * RPW);  // first row, within the group
  const int64_t slot = slots ? slots[b] : b;
  const bool live = slot >= 0 && slot < nslots;
  const int64_t R = (int64_t)d.H * d.P;

  float* const st = state + (slot * R + (int64_t)g * d.RG + q0 + seg) * d.N + sl * V;
  const int step = RPW * d.N;        // floats from a lane's row to its next
  const int rows = d.RG - q0 - seg;  // row i of the lane exists while i * RPW < rows
  Raw<float, V> raw[RB][NV];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int n = 0; n < NV; ++n)
      raw[i][n] = live && i * RPW < rows && (n * LPR + sl) * V < d.N
                      ? ld_raw<float, V>(st + (int64_t)i * step + n * LPR * V)
                      : zero_raw<float, V>();

  // this lane's own row (lanes sl < RB)
  const int qm = q0 + sl * RPW + seg;
  const bool mine = sl < RB && qm < d.RG;
  const int64_t rm = (int64_t)g * d.RG + qm;
  float a = 0.f, bb = 0.f, val = 0.f;
  if (mine && live) {
    const int h = (int)(rm / d.P);
    val = to_f(v[b * d.vs + rm]);
    a = decay(softplus(to_f(dt[(int64_t)b * d.H + h]) + (dt_bias ? dt_bias[h] : 0.f)), A[h] * kLog2e);
    bb = sigmoid(to_f(beta[(int64_t)b * d.H + h]));
  }
  float out = 0.f;
  if (live) {
    const Tin* kp = k + b * d.ks + (int64_t)g * d.N + sl * V;
    const Tin* qp = q + b * d.qs + (int64_t)g * d.N + sl * V;
    float kv[NV][V], qv[NV][V], kq = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = (n * LPR + sl) * V + j < d.N;
        kv[n][j] = in ? to_f(kp[n * LPR * V + j]) : 0.f;
        qv[n][j] = in ? to_f(qp[n * LPR * V + j]) : 0.f;
        kq = fmaf(kv[n][j], qv[n][j], kq);
      }
    float sk[RB], sq[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      sk[i] = sq[i] = 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        float s[V];
        unpack<float, V>(raw[i][n], s);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sk[i] = fmaf(s[j], kv[n][j], sk[i]);
          sq[i] = fmaf(s[j], qv[n][j], sq[i]);
        }
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      kq += __shfl_xor_sync(0xffffffffu, kq, o);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], o);
        sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
      }
    }
    float mk = 0.f, mq = 0.f;
#pragma unroll
    for (int i = 0; i < RB; ++i)
      if (sl == i) mk = sk[i], mq = sq[i];
    const float u = bb * fmaf(-a, mk, val);
    out = d.scale * fmaf(u, kq, a * mq);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const float ai = __shfl_sync(0xffffffffu, a, i, LPR), ui = __shfl_sync(0xffffffffu, u, i, LPR);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        float s[V];
        unpack<float, V>(raw[i][n], s);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = fmaf(ai, s[j], ui * kv[n][j]);
        if (i * RPW < rows && (n * LPR + sl) * V < d.N)
          st_raw<float, V>(st + (int64_t)i * step + n * LPR * V, pack<float, V>(s));
      }
    }
  }
  if (mine) y[(int64_t)b * R + rm] = from_f<Tout>(live ? out : 0.f);
}

struct DeltaStepPtrs {
  const void *q, *k, *v, *dt;
  const float *dt_bias, *A;
  const void* beta;
  float* state;
  const int* slots;
  int64_t nslots;
  void* y;
};

template <typename Tin, typename Tout, int LPR, int V, int NV, int RB>
int launch_step(DeltaStepDims d, const DeltaStepPtrs& p, cudaStream_t s) {
  const int rows = RB * (32 / LPR);
  d.tiles = (d.RG + rows - 1) / rows;
  const int64_t blocks = ((int64_t)d.B * d.G * d.tiles + kStepWarps - 1) / kStepWarps;
  if (blocks > 0x7fffffff) return SSD_ERR_UNSUPPORTED;
  SSD_LAUNCH("k_delta_step", s,
             k_delta_step<Tin, Tout, LPR, V, NV, RB><<<(unsigned)blocks, 32 * kStepWarps, 0, s>>>(
                 static_cast<const Tin*>(p.q), static_cast<const Tin*>(p.k),
                 static_cast<const Tin*>(p.v), static_cast<const Tin*>(p.dt), p.dt_bias, p.A,
                 static_cast<const Tin*>(p.beta), p.state, p.slots, p.nslots,
                 static_cast<Tout*>(p.y), d));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// Lanes of a row: the power of two that covers its V-wide pieces, from 8 on; a row of
// more than 32 pieces takes several a lane.  Rows of a lane: 8, to have 128 bytes a lane
// in flight; 4 where the states are under 32 MB and more warps count for more.  Measured
// with 128 key columns, us a call in a row of them, 4 and 8 rows a lane: 2048 state rows
// 2.42 and 2.57, 16384 3.92 and 4.16, 32768 4.63 and 4.60, 65536 9.52 and 9.15, 131072
// 16.6 and 15.6; with 64: 65536 5.65 and 6.00, 131072 9.13 and 8.88.
// Fewer where a row takes several pieces a lane, whose registers they share.
template <typename Tin, typename Tout>
int pick_step(const DeltaStepDims& d, const DeltaStepPtrs& p, bool vec, cudaStream_t s) {
  const int nv = vec ? d.N / 4 : d.N;
  const int lpr = nv > 16 ? 32 : nv > 8 ? 16 : 8;
  const bool few = (int64_t)d.B * d.H * d.P * lpr < (int64_t)65536 * 32;
  if (!vec) {  // rows that fill no 16 bytes
    if (nv > 64) return launch_step<Tin, Tout, 32, 1, 8, 2>(d, p, s);
    return launch_step<Tin, Tout, 32, 1, 2, 4>(d, p, s);
  }
  if (nv > 32) return launch_step<Tin, Tout, 32, 4, 2, 4>(d, p, s);
  if (lpr == 32)
    return few ? launch_step<Tin, Tout, 32, 4, 1, 4>(d, p, s)
               : launch_step<Tin, Tout, 32, 4, 1, 8>(d, p, s);
  if (lpr == 16)
    return few ? launch_step<Tin, Tout, 16, 4, 1, 4>(d, p, s)
               : launch_step<Tin, Tout, 16, 4, 1, 8>(d, p, s);
  return few ? launch_step<Tin, Tout, 8, 4, 1, 4>(d, p, s)
             : launch_step<Tin, Tout, 8, 4, 1, 8>(d, p, s);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_gated_delta_step(const ssd_delta_shape* sh, const void* q, const void* k, const void* v,
                         const void* dt, const float* dt_bias, const float* A, const void* beta,
                         float* state, const int32_t* slots, int64_t nslots, void* y,
                         void* stream) {
  if (!sh || sh->batch < 1 || sh->seqlen != 1 || sh->nheads < 1 || sh->headdim < 1 ||
      sh->dstate < 1 || sh->ngroups < 1 || sh->nheads % sh->ngroups != 0)
    return SSD_ERR_INVALID_ARG;
  if ((sh->in_dtype != SSD_F32 && sh->in_dtype != SSD_BF16) ||
      (sh->out_dtype != SSD_F32 && sh->out_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  const int64_t gn = sh->ngroups * sh->dstate, hp = sh->nheads * sh->headdim;
  if ((sh->q_row_stride && sh->q_row_stride < gn) || (sh->k_row_stride && sh->k_row_stride < gn) ||
      (sh->v_row_stride && sh->v_row_stride < hp))
    return SSD_ERR_INVALID_ARG;
  if (nslots < 1 || (!slots && nslots < sh->batch)) return SSD_ERR_INVALID_ARG;
  if (!q || !k || !v || !dt || !A || !beta || !state || !y) return SSD_ERR_INVALID_ARG;
  if (sh->batch >= (1 << 24) || sh->nheads >= (1 << 20) || sh->headdim >= (1 << 14) ||
      sh->dstate > 256 || hp >= (1 << 26))
    return SSD_ERR_UNSUPPORTED;
  if (sh->in_dtype == SSD_F32 && sh->out_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  const bool ib = sh->in_dtype == SSD_BF16, ob = sh->out_dtype == SSD_BF16;
  const uintptr_t im = ib ? 1 : 3, om = ob ? 1 : 3;
  auto off = [](const void* x, uintptr_t m) { return (reinterpret_cast<uintptr_t>(x) & m) != 0; };
  if (off(q, im) || off(k, im) || off(v, im) || off(dt, im) || off(beta, im) || off(y, om) ||
      off(dt_bias, 3) || off(A, 3) || off(state, 3) || off(slots, 3))
    return SSD_ERR_INVALID_ARG;
  DeltaStepDims d{};
  d.B = (int)sh->batch, d.H = (int)sh->nheads, d.G = (int)sh->ngroups;
  d.P = (int)sh->headdim, d.N = (int)sh->dstate, d.RG = (int)(hp / sh->ngroups);
  d.qs = sh->q_row_stride ? sh->q_row_stride : gn;
  d.ks = sh->k_row_stride ? sh->k_row_stride : gn;
  d.vs = sh->v_row_stride ? sh->v_row_stride : hp;
  d.scale = sh->scale;
  const DeltaStepPtrs p{q, k, v, dt, dt_bias, A, beta, state, slots, nslots, y};
  const bool vec = vec_ok(state, d.N, 4, 4) && d.N % 4 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (ib && ob) return pick_step<bf16, bf16>(d, p, vec, s);
  if (ib) return pick_step<bf16, float>(d, p, vec, s);
  return pick_step<float, float>(d, p, vec, s);
}

}  // extern "C"
