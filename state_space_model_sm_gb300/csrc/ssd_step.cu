// One token of the scan, for decoding: the carried state moves by one step
// of the recurrence and gives the token's output,
//     delta = softplus(dt + dt_bias),  h <- exp(delta A) h + delta x B,
//     y = C . h + D x
// for the SSD scan (one decay per head, state rows (head, p)) and for the
// selective scan (a decay per channel and state, state rows = channels, and
// the optional gate y silu(z)).  The state lives in a cache of slots; a batch
// row names its slot.
//
// The state is read and written once, 8 bytes per 6 operations (and, in the
// selective form, one exponential): HBM-bound.  A row's N states lie across
// the LPR lanes of a warp segment, V per lane (a 16-byte access), so a warp
// streams whole 512-byte lines; each lane holds RB rows' states at once, and
// they are the first thing loaded, so that the latency of what a row needs once
// (softplus, decay, skip term, gate: computed by one lane of its segment and
// broadcast) lies under theirs; five blocks an SM.  171 us for 256 batch rows of
// 64 x 64 x 128 states: 6.3 TB/s, 0.93 of a plain copy's rate (203 us before the
// states were loaded first).  A single row's call is its launch: 2.3 us in a
// captured graph.
#include <cuda_bf16.h>

#include "layer_math.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace lm;
using bf16 = __nv_bfloat16;

struct StepDims {
  int B, R, P, N, G;  // batch rows; state rows of each, P to a head; states; groups
  int RG;             // state rows of a group: R / G
  int tiles;          // warp tiles of a group
  int64_t xs, dts, bs, cs, zs;  // elements between batch rows
};

constexpr int kStepWarps = 4;

// SEL: the selective form (A is (R, N); P = 1).
template <typename Tin, typename Tout, bool SEL, int LPR, int V, int RB>
__global__ void __launch_bounds__(32 * kStepWarps, RB > 2 ? 5 : 1)
    k_step(const Tin* __restrict__ x, const Tin* __restrict__ dt, const float* __restrict__ dt_bias,
           const float* __restrict__ A, const Tin* __restrict__ Bm, const Tin* __restrict__ Cm,
           const float* __restrict__ D, const Tin* __restrict__ z, float* __restrict__ state,
           const int* __restrict__ slots, int64_t nslots, Tout* __restrict__ y, StepDims d) {
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

  // the states of the rows' first V x LPR columns, ahead of everything else: the
  // scalars below are loaded and formed while they are in flight
  float* const st = state + (slot * d.R + (int64_t)g * d.RG + q0 + seg) * d.N + sl * V;
  const float* const ap = SEL ? A + ((int64_t)g * d.RG + q0 + seg) * d.N + sl * V : nullptr;
  const int step = RPW * d.N;      // floats from a lane's row to its next
  const int rows = d.RG - q0 - seg;  // row i of the lane exists while i * RPW < rows
  Raw<float, V> raw[RB], ra[RB];
  auto fetch = [&](int n) {  // columns sl * V + n ..
    const bool in = live && sl * V + n < d.N;  // V divides N where V > 1
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const bool ok = in && i * RPW < rows;
      raw[i] = ok ? ld_raw<float, V>(st + (int64_t)i * step + n) : zero_raw<float, V>();
      if constexpr (SEL) ra[i] = ok ? ld_raw<float, V>(ap + (int64_t)i * step + n) : zero_raw<float, V>();
    }
  };
  fetch(0);

  // this lane's own row (lanes sl < RB): what the row needs once
  const int qm = q0 + sl * RPW + seg;
  const bool mine = sl < RB && qm < d.RG;
  const int rm = g * d.RG + qm;
  float delta = 0.f, dec = 0.f, dtx = 0.f, skip = 0.f;
  if (mine && live) {
    const int hd = SEL ? rm : rm / d.P;
    const float xv = to_f(x[b * d.xs + rm]);
    delta = softplus(to_f(dt[b * d.dts + hd]) + (dt_bias ? dt_bias[hd] : 0.f));
    if constexpr (!SEL) dec = decay(delta, A[hd] * kLog2e);
    dtx = delta * xv;
    skip = D ? D[hd] * xv : 0.f;
  }

  float acc[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) acc[i] = 0.f;
  if (live) {
    const Tin* bp = Bm + b * d.bs + (int64_t)g * d.N + sl * V;
    const Tin* cp = Cm + b * d.cs + (int64_t)g * d.N + sl * V;
    for (int n = 0; n < d.N; n += LPR * V) {
      if (n > 0) fetch(n);
      const bool in = sl * V + n < d.N;
      float bv[V], cv[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        bv[j] = in ? to_f(bp[n + j]) : 0.f;
        cv[j] = in ? to_f(cp[n + j]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const float dx = __shfl_sync(0xffffffffu, dtx, i, LPR);
        float h[V], a[V];
        unpack<float, V>(raw[i], h);
        if constexpr (SEL) {
          const float dl = __shfl_sync(0xffffffffu, delta, i, LPR);
          unpack<float, V>(ra[i], a);
#pragma unroll
          for (int j = 0; j < V; ++j) a[j] = decay(dl, a[j] * kLog2e);
        } else {
          const float dc = __shfl_sync(0xffffffffu, dec, i, LPR);
#pragma unroll
          for (int j = 0; j < V; ++j) a[j] = dc;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          h[j] = fmaf(a[j], h[j], dx * bv[j]);
          acc[i] = fmaf(cv[j], h[j], acc[i]);
        }
        if (in && i * RPW < rows) st_raw<float, V>(st + (int64_t)i * step + n, pack<float, V>(h));
      }
    }
  }
  float out = 0.f;
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    float v = acc[i];
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (sl == i) out = v;
  }
  if (mine) {
    out += skip;
    if (SEL && z && live) {
      const float zv = to_f(z[b * d.zs + rm]);
      out *= zv * sigmoid(zv);
    }
    y[(int64_t)b * d.R + rm] = from_f<Tout>(live ? out : 0.f);
  }
}

struct StepPtrs {
  const void *x, *dt;
  const float *dt_bias, *A;
  const void *B, *C;
  const float* D;
  const void* z;
  float* state;
  const int* slots;
  int64_t nslots;
  void* y;
};

template <typename Tin, typename Tout, bool SEL, int LPR, int V, int RB>
int launch_step(StepDims d, const StepPtrs& p, cudaStream_t s) {
  const int rows = RB * (32 / LPR);
  d.tiles = (d.RG + rows - 1) / rows;
  const int64_t blocks = ((int64_t)d.B * d.G * d.tiles + kStepWarps - 1) / kStepWarps;
  if (blocks > 0x7fffffff) return SSD_ERR_UNSUPPORTED;
  SSD_LAUNCH(SEL ? "k_selective_step" : "k_ssd_step", s,
             k_step<Tin, Tout, SEL, LPR, V, RB><<<(unsigned)blocks, 32 * kStepWarps, 0, s>>>(
                 static_cast<const Tin*>(p.x), static_cast<const Tin*>(p.dt), p.dt_bias, p.A,
                 static_cast<const Tin*>(p.B), static_cast<const Tin*>(p.C), p.D,
                 static_cast<const Tin*>(p.z), p.state, p.slots, p.nslots,
                 static_cast<Tout*>(p.y), d));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// Lanes per row: the power of two that covers the row's V-wide vectors, 32 at
// most (then the row is walked).  Rows per lane: 8, to have 128 bytes a lane in
// flight (171 us at 256 rows of 64 x 64 x 128 states, 240 with 2); 2 where 8 would
// leave fewer than two warps per SM quarter (one row of 24 x 64 x 128: 2.3 us, 2.6
// with 8).  4 in rows of four lanes, whatever the size (16 rows of 4096 x 16: 3.6 us,
// 3.8 with 2), and in the selective form in place of 8 where a lane's access is 4
// states, since it holds as many of A (256 rows of 4096 x 64: 127 us, and 138 with 8,
// which spill; 64 rows of 4096 x 32: 12.8 and 20.3).
template <typename Tin, typename Tout, bool SEL, int V>
int pick_step(const StepDims& d, const StepPtrs& p, cudaStream_t s) {
  const int nv = (d.N + V - 1) / V;
  const int lpr = nv > 16 ? 32 : nv > 8 ? 16 : nv > 4 ? 8 : nv > 2 ? 4 : nv > 1 ? 2 : 1;
  constexpr int many = SEL && V == 4 ? 4 : 8;
  const bool few = (int64_t)d.B * d.R * lpr < (int64_t)152 * 8 * 32 * 8;
  switch (lpr) {
    case 1: return launch_step<Tin, Tout, SEL, 1, V, 1>(d, p, s);
    case 2: return launch_step<Tin, Tout, SEL, 2, V, 2>(d, p, s);
    case 4: return launch_step<Tin, Tout, SEL, 4, V, 4>(d, p, s);
    case 8:
      return few ? launch_step<Tin, Tout, SEL, 8, V, 2>(d, p, s)
                 : launch_step<Tin, Tout, SEL, 8, V, many>(d, p, s);
    case 16:
      return few ? launch_step<Tin, Tout, SEL, 16, V, 2>(d, p, s)
                 : launch_step<Tin, Tout, SEL, 16, V, many>(d, p, s);
    default:
      return few ? launch_step<Tin, Tout, SEL, 32, V, 2>(d, p, s)
                 : launch_step<Tin, Tout, SEL, 32, V, many>(d, p, s);
  }
}

template <bool SEL>
int run_step(const StepDims& d, int in_dtype, int out_dtype, const StepPtrs& p, cudaStream_t s) {
  const bool ib = in_dtype == SSD_BF16, ob = out_dtype == SSD_BF16;
  const uintptr_t im = ib ? 1 : 3, om = ob ? 1 : 3;
  auto off = [](const void* q, uintptr_t m) { return (reinterpret_cast<uintptr_t>(q) & m) != 0; };
  if (off(p.x, im) || off(p.dt, im) || off(p.B, im) || off(p.C, im) || off(p.z, im) ||
      off(p.y, om) || off(p.dt_bias, 3) || off(p.A, 3) || off(p.D, 3) || off(p.state, 3) ||
      off(p.slots, 3))
    return SSD_ERR_INVALID_ARG;
  const bool vec = d.N % 4 == 0 && vec_ok(p.state, d.N, 4, 4) && (!SEL || vec_ok(p.A, d.N, 4, 4));
  if (ib && ob) return vec ? pick_step<bf16, bf16, SEL, 4>(d, p, s) : pick_step<bf16, bf16, SEL, 1>(d, p, s);
  if (ib) return vec ? pick_step<bf16, float, SEL, 4>(d, p, s) : pick_step<bf16, float, SEL, 1>(d, p, s);
  return vec ? pick_step<float, float, SEL, 4>(d, p, s) : pick_step<float, float, SEL, 1>(d, p, s);
}

bool dtypes_ok(int in, int out) {
  return (in == SSD_F32 || in == SSD_BF16) && (out == SSD_F32 || out == SSD_BF16);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_step(const ssd_shape* sh, const void* x, const void* dt, const float* dt_bias,
             const float* A, const void* B, const void* C, const float* D, float* state,
             const int32_t* slots, int64_t nslots, void* y, void* stream) {
  if (!sh || sh->batch < 1 || sh->nheads < 1 || sh->headdim < 1 || sh->dstate < 1 ||
      sh->ngroups < 1 || sh->nheads % sh->ngroups != 0 || !dtypes_ok(sh->in_dtype, sh->out_dtype))
    return SSD_ERR_INVALID_ARG;
  if (nslots < 1 || (!slots && nslots < sh->batch)) return SSD_ERR_INVALID_ARG;
  if (!x || !dt || !A || !B || !C || !state || !y) return SSD_ERR_INVALID_ARG;
  if (sh->batch >= (1 << 24) || sh->nheads >= (1 << 20) || sh->headdim > (1 << 14) ||
      sh->headdim * sh->dstate > 16384 || sh->nheads * sh->headdim >= (1 << 26))
    return SSD_ERR_UNSUPPORTED;
  if (sh->in_dtype == SSD_F32 && sh->out_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  StepDims d{};
  d.B = (int)sh->batch, d.P = (int)sh->headdim, d.N = (int)sh->dstate, d.G = (int)sh->ngroups;
  d.R = (int)(sh->nheads * sh->headdim), d.RG = d.R / d.G;
  d.xs = d.R, d.dts = sh->nheads, d.bs = d.cs = (int64_t)d.G * d.N;
  const StepPtrs p{x, dt, dt_bias, A, B, C, D, nullptr, state, slots, nslots, y};
  return run_step<false>(d, sh->in_dtype, sh->out_dtype, p, static_cast<cudaStream_t>(stream));
}

int ssd_selective_step(const ssd_selective_shape* sh, const void* x, const void* dt,
                       const float* dt_bias, const float* A, const void* B, const void* C,
                       const float* D, const void* z, float* state, const int32_t* slots,
                       int64_t nslots, void* y, void* stream) {
  if (!sh || sh->batch < 1 || sh->seqlen != 1 || sh->channels < 1 || sh->dstate < 1 ||
      sh->ngroups < 1 || sh->channels % sh->ngroups != 0 ||
      !dtypes_ok(sh->in_dtype, sh->out_dtype))
    return SSD_ERR_INVALID_ARG;
  const int64_t gn = sh->ngroups * sh->dstate;
  if ((sh->z_row_stride && sh->z_row_stride < sh->channels) ||
      (sh->b_row_stride && sh->b_row_stride < gn) || (sh->c_row_stride && sh->c_row_stride < gn))
    return SSD_ERR_INVALID_ARG;
  if (nslots < 1 || (!slots && nslots < sh->batch)) return SSD_ERR_INVALID_ARG;
  if (!x || !dt || !A || !B || !C || !state || !y) return SSD_ERR_INVALID_ARG;
  if (sh->batch >= (1 << 24) || sh->channels >= (1 << 24) || sh->dstate > 256)
    return SSD_ERR_UNSUPPORTED;
  if (sh->in_dtype == SSD_F32 && sh->out_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  StepDims d{};
  d.B = (int)sh->batch, d.R = (int)sh->channels, d.P = 1, d.N = (int)sh->dstate;
  d.G = (int)sh->ngroups, d.RG = d.R / d.G;
  d.xs = d.dts = d.R;
  d.bs = sh->b_row_stride ? sh->b_row_stride : gn, d.cs = sh->c_row_stride ? sh->c_row_stride : gn;
  d.zs = sh->z_row_stride ? sh->z_row_stride : d.R;
  const StepPtrs p{x, dt, dt_bias, A, B, C, D, z, state, slots, nslots, y};
  return run_step<true>(d, sh->in_dtype, sh->out_dtype, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
