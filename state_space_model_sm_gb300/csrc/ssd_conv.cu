// Short causal depthwise convolution, the step in front of a layer's scan:
//     u[t, c] = bias[c] + sum_{k < K} w[c, k] x[t - K + 1 + k, c]
//     y = silu(u) or u,  silu(u) = u / (1 + e^-u)
// with x before position 0 taken from the carried state (the K - 1 inputs
// before the sequence, oldest first) or 0; its backward; and the single-token
// form, which shifts the state by one.  The pages name no kernel for it.
//
// All three are HBM streams: an element costs 2 K + ~8 operations against 4
// to 8 bytes, far below the machine's ratio.  Channels are contiguous, so a
// thread owns V consecutive channels (one 16-byte access; 8-byte in the bf16
// backward, whose live set is three times the forward's) and walks positions
// with the last K - 1 inputs in registers: every input is read once, plus
// K - 1 rows per segment.
#include <cuda_bf16.h>

#include "layer_math.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace lm;
using bf16 = __nv_bfloat16;

struct ConvDims {
  int B, T, C, nvec;      // nvec: vectors of channels a row
  int64_t xs, xb;         // elements between x's positions, and its batch rows
  int seg, nseg;          // positions a thread walks; segments a sequence
  int silu;
};

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// Row t of the sequence's inputs, t >= -(K - 1): the carried state before 0.
template <typename T, int V, int K>
__device__ __forceinline__ Raw<T, V> ld_x(const T* x, const T* init, const ConvDims& d, int t) {
  if (t >= 0) return ld_raw<T, V>(x + (int64_t)t * d.xs);
  if (init) return ld_raw<T, V>(init + (int64_t)(t + K - 1) * d.C);
  return zero_raw<T, V>();
}

// Thread: V channels of one segment.  Work items are (batch, segment, vector)
// with the vector fastest, so a warp's accesses are contiguous.  kU positions
// are loaded before they are used.
constexpr int kU = 8;

template <typename Tin, typename Tout, int V, int K>
__global__ void __launch_bounds__(256)
    k_conv_fwd(const Tin* __restrict__ x, const float* __restrict__ w,
               const float* __restrict__ bias, const Tin* __restrict__ init,
               const int* __restrict__ lengths, Tout* __restrict__ y, Tin* __restrict__ final_state,
               ConvDims d) {
  const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t per_b = (int64_t)d.nseg * d.nvec;
  const int b = (int)(item / per_b);
  if (b >= d.B) return;
  const int rem = (int)(item - b * per_b), s = rem / d.nvec, c0 = (rem - s * d.nvec) * V;
  const int n = clamp_len(lengths, b, d.T);
  x += b * d.xb + c0;
  if (init) init += (int64_t)b * (K - 1) * d.C + c0;
  y += (int64_t)b * d.T * d.C + c0;

  if (s == 0 && final_state) {
    Tin* f = final_state + (int64_t)b * (K - 1) * d.C + c0;
    for (int j = 0; j < K - 1; ++j)
      st_raw<Tin, V>(f + (int64_t)j * d.C, ld_x<Tin, V, K>(x, init, d, n - (K - 1) + j));
  }

  float wk[K][V], bs[V], win[K][V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) wk[k][i] = w[(int64_t)(c0 + i) * K + k];
    bs[i] = bias ? bias[c0 + i] : 0.f;
  }
  const int t0 = s * d.seg, t1 = min(d.T, t0 + d.seg), tv = min(t1, n);
#pragma unroll
  for (int k = 0; k < K - 1; ++k)
    unpack<Tin, V>(ld_x<Tin, V, K>(x, init, d, min(t0, d.T) - (K - 1) + k), win[k + 1]);
  for (int tb = t0; tb < tv; tb += kU) {
    Raw<Tin, V> raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      raw[u] = tb + u < tv ? ld_raw<Tin, V>(x + (int64_t)(tb + u) * d.xs) : zero_raw<Tin, V>();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i];
      unpack<Tin, V>(raw[u], win[K - 1]);
      if (tb + u < tv) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float a = bs[i];
#pragma unroll
          for (int k = 0; k < K; ++k) a = fmaf(wk[k][i], win[k][i], a);
          o[i] = d.silu ? a * sigmoid(a) : a;
        }
        st_raw<Tout, V>(y + (int64_t)(tb + u) * d.C, pack<Tout, V>(o));
      }
    }
  }
  for (int t = max(t0, n); t < t1; ++t) st_raw<Tout, V>(y + (int64_t)t * d.C, zero_raw<Tout, V>());
}

// Backward.  With du = dy silu'(u) (0 from the sequence's length on),
//     dx[s] = sum_k w[k] du[s + K - 1 - k]  (+ dfinal where x[s] is carried on)
//     dw[k] = sum_t du[t] x[t - K + 1 + k],  dbias = sum_t du[t].
// A warp owns 32 vectors of channels and one segment, whose du it forms for
// K - 1 positions past the end as well, so dx needs no second pass; the dw
// sums stay in registers, are added over the block's warps in shared memory
// and written as one partial per block, which k_conv_dw adds in order.
constexpr int kBwdWarps = 8;

template <typename Tin, typename Tout, int V, int K>
__global__ void __launch_bounds__(32 * kBwdWarps)
    k_conv_bwd(const Tin* __restrict__ x, const float* __restrict__ w,
               const float* __restrict__ bias, const Tin* __restrict__ init,
               const int* __restrict__ lengths, const Tin* __restrict__ dy,
               const Tin* __restrict__ dfinal, Tout* __restrict__ dx, Tout* __restrict__ dinit,
               float* __restrict__ part, ConvDims d, int nblk) {
  __shared__ float red[kBwdWarps][K + 1][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v = blockIdx.x * 32 + lane, c0 = v * V;
  const int b = blockIdx.y / nblk, s = (blockIdx.y - b * nblk) * kBwdWarps + warp;
  float dw[K + 1][V];
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = 0.f;

  if (v < d.nvec && s < d.nseg) {
    const int n = clamp_len(lengths, b, d.T);
    x += b * d.xb + c0;
    dy += (int64_t)b * d.T * d.C + c0;
    dx += (int64_t)b * d.T * d.C + c0;
    const int64_t st0 = (int64_t)b * (K - 1) * d.C + c0;
    if (init) init += st0;
    float wk[K][V], bs[V], win[K][V], du[K][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        wk[k][i] = w[(int64_t)(c0 + i) * K + k];
        du[k][i] = 0.f;
      }
      bs[i] = bias ? bias[c0 + i] : 0.f;
    }
    const int t0 = s * d.seg, t1 = min(d.T, t0 + d.seg);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      unpack<Tin, V>(ld_x<Tin, V, K>(x, init, d, t0 - (K - 1) + k), win[k + 1]);
    const int te = t1 + K - 1;  // one past the last du this segment needs
    constexpr int U = 4;
    for (int tb = t0; tb < te; tb += U) {
      Raw<Tin, V> rx[U], rg[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = tb + u < min(te, n);
        rx[u] = in ? ld_raw<Tin, V>(x + (int64_t)(tb + u) * d.xs) : zero_raw<Tin, V>();
        rg[u] = in ? ld_raw<Tin, V>(dy + (int64_t)(tb + u) * d.C) : zero_raw<Tin, V>();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u;
        if (t < te) {
          float g[V];
#pragma unroll
          for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i], du[k][i] = du[k + 1][i];
          unpack<Tin, V>(rx[u], win[K - 1]);
          unpack<Tin, V>(rg[u], g);
          const bool in = t < n;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (d.silu) {
              float a = bs[i];
#pragma unroll
              for (int k = 0; k < K; ++k) a = fmaf(wk[k][i], win[k][i], a);
              const float sg = sigmoid(a);
              g[i] *= sg * (1.f + a * (1.f - sg));
            }
            du[K - 1][i] = in ? g[i] : 0.f;
          }
          if (in && t < t1) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
              for (int k = 0; k < K; ++k) dw[k][i] = fmaf(du[K - 1][i], win[k][i], dw[k][i]);
              dw[K][i] += du[K - 1][i];
            }
          }
          const int sp = t - (K - 1);  // dx of this position is complete now
          if (sp >= t0 || s == 0) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
              o[i] = 0.f;
#pragma unroll
              for (int k = 0; k < K; ++k) o[i] = fmaf(wk[k][i], du[K - 1 - k][i], o[i]);
            }
            const int j = t - n;  // x[sp] is entry j of the final state
            if (dfinal && j >= 0 && j < K - 1) {
              float f[V];
              unpack<Tin, V>(ld_raw<Tin, V>(dfinal + st0 + (int64_t)j * d.C), f);
#pragma unroll
              for (int i = 0; i < V; ++i) o[i] += f[i];
            }
            if (sp >= 0)
              st_raw<Tout, V>(dx + (int64_t)sp * d.C, pack<Tout, V>(o));
            else if (dinit)
              st_raw<Tout, V>(dinit + st0 + (int64_t)t * d.C, pack<Tout, V>(o));
          }
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][k][lane * V + i] = dw[k][i];
  __syncthreads();
  // part (blocks, K + 1, C)
  const int nc = min(32 * V, d.C - blockIdx.x * 32 * V);
  float* p = part + (int64_t)blockIdx.y * (K + 1) * d.C + (int64_t)blockIdx.x * 32 * V;
  for (int i = threadIdx.x; i < (K + 1) * 32 * V; i += blockDim.x) {
    const int k = i / (32 * V), c = i - k * (32 * V);
    if (c < nc) {
      float a = 0.f;
#pragma unroll
      for (int wv = 0; wv < kBwdWarps; ++wv) a += red[wv][k][c];
      p[(int64_t)k * d.C + c] = a;
    }
  }
}

// dw (C, K) and dbias (C) from the blocks' partials: a block owns 32
// channels of one tap, its 8 warps take every 8th partial.
__global__ void __launch_bounds__(256)
    k_conv_dw(const float* __restrict__ part, float* __restrict__ dw, float* __restrict__ dbias,
              int nparts, int C, int K) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
  float a = 0.f;
  if (c < C)
    for (int i = warp; i < nparts; i += 8) a += part[((int64_t)i * (K + 1) + k) * C + c];
  red[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < C) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][lane];
    if (k < K)
      dw[(int64_t)c * K + k] = t;
    else if (dbias)
      dbias[c] = t;
  }
}

// One token: thread = V channels of one batch row; its state is read, used
// and written back shifted by one.
template <typename Tin, typename Tout, int V, int K>
__global__ void __launch_bounds__(128)
    k_conv_step(const Tin* __restrict__ x, Tin* __restrict__ state, const float* __restrict__ w,
                const float* __restrict__ bias, const int* __restrict__ slots, int64_t nslots,
                Tout* __restrict__ y, ConvDims d) {
  const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int b = (int)(item / d.nvec), c0 = (int)(item - (int64_t)b * d.nvec) * V;
  if (b >= d.B) return;
  const int64_t slot = slots ? slots[b] : b;
  Tout* yo = y + (int64_t)b * d.C + c0;
  if (slot < 0 || slot >= nslots) {
    st_raw<Tout, V>(yo, zero_raw<Tout, V>());
    return;
  }
  Tin* st = state + slot * (K - 1) * d.C + c0;
  Raw<Tin, V> raw[K];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) raw[k] = ld_raw<Tin, V>(st + (int64_t)k * d.C);
  raw[K - 1] = ld_raw<Tin, V>(x + (int64_t)b * d.xs + c0);
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = bias ? bias[c0 + i] : 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float f[V];
    unpack<Tin, V>(raw[k], f);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(w[(int64_t)(c0 + i) * K + k], f[i], o[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (d.silu) o[i] *= sigmoid(o[i]);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) st_raw<Tin, V>(st + (int64_t)k * d.C, raw[k + 1]);
  st_raw<Tout, V>(yo, pack<Tout, V>(o));
}

// ------------------------------------------------------------------- host

int conv_dims(const ssd_conv_shape* s, ConvDims* d) {
  if (!s || s->batch < 1 || s->seqlen < 1 || s->channels < 1 || s->width < 1)
    return SSD_ERR_INVALID_ARG;
  if ((s->in_dtype != SSD_F32 && s->in_dtype != SSD_BF16) ||
      (s->out_dtype != SSD_F32 && s->out_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  if ((s->x_row_stride != 0 && s->x_row_stride < s->channels) || s->x_batch_stride < 0)
    return SSD_ERR_INVALID_ARG;
  if (s->width < 2 || s->width > 4) return SSD_ERR_UNSUPPORTED;
  if (s->in_dtype == SSD_F32 && s->out_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->batch >= 65536 || s->seqlen >= (1 << 30) || s->channels >= (1 << 24))
    return SSD_ERR_UNSUPPORTED;
  d->B = (int)s->batch, d->T = (int)s->seqlen, d->C = (int)s->channels;
  d->xs = s->x_row_stride ? s->x_row_stride : s->channels;
  d->xb = s->x_row_stride ? s->x_batch_stride : d->xs * d->T;
  d->silu = s->silu != 0;
  return SSD_OK;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Positions a forward thread walks: 32 reads 3 extra rows (from L2) in 32;
// short inputs take shorter segments, down to 8, until the grid holds about
// one wave of threads.
void fwd_segments(ConvDims* d) {
  d->seg = 32;
  while (d->seg > kU && (int64_t)d->B * ceil_div(d->T, d->seg) * d->nvec < 152 * 1024) d->seg /= 2;
  d->nseg = ceil_div(d->T, d->seg);
}

// The backward forms du for K - 1 positions past each segment: 32 positions
// keep that under a tenth; shorter ones, down to 8, while the blocks (32
// vectors x 8 segments) would not fill the SMs.
void bwd_segments(ConvDims* d) {
  d->seg = 32;
  while (d->seg > 8 && (int64_t)d->B * ceil_div(d->T, d->seg * kBwdWarps) * ceil_div(d->nvec, 32) <
                           3 * 152)
    d->seg /= 2;
  d->nseg = ceil_div(d->T, d->seg);
}

// the backward's vector width and its blocks per sequence: shape-only, so
// the workspace query and the call agree
int bwd_parts(const ConvDims& d) { return d.B * ceil_div(d.nseg, kBwdWarps); }

template <typename Tin, typename Tout, int V>
int launch_fwd(ConvDims d, int K, const void* x, const float* w, const float* bias,
               const void* init, const int* lengths, void* y, void* final_state, cudaStream_t s) {
  d.nvec = d.C / V;
  fwd_segments(&d);
  const int64_t items = (int64_t)d.B * d.nseg * d.nvec, blocks = (items + 255) / 256;
  if (blocks > 0x7fffffff) return SSD_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    SSD_LAUNCH("k_conv_fwd", s,
               kern<<<(unsigned)blocks, 256, 0, s>>>(
                   static_cast<const Tin*>(x), w, bias, static_cast<const Tin*>(init), lengths,
                   static_cast<Tout*>(y), static_cast<Tin*>(final_state), d));
  };
  if (K == 2) go(k_conv_fwd<Tin, Tout, V, 2>);
  if (K == 3) go(k_conv_fwd<Tin, Tout, V, 3>);
  if (K == 4) go(k_conv_fwd<Tin, Tout, V, 4>);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

template <typename Tin, typename Tout, int V>
int launch_bwd(ConvDims d, int K, const void* x, const float* w, const float* bias,
               const void* init, const int* lengths, const void* dy, const void* dfinal, void* dx,
               float* dw, float* dbias, void* dinit, float* part, cudaStream_t s) {
  d.nvec = d.C / V;
  const int nblk = ceil_div(d.nseg, kBwdWarps), nparts = bwd_parts(d);
  const dim3 grid(ceil_div(d.nvec, 32), nparts);
  auto go = [&](auto kern) {
    SSD_LAUNCH("k_conv_bwd", s,
               kern<<<grid, 32 * kBwdWarps, 0, s>>>(
                   static_cast<const Tin*>(x), w, bias, static_cast<const Tin*>(init), lengths,
                   static_cast<const Tin*>(dy), static_cast<const Tin*>(dfinal),
                   static_cast<Tout*>(dx), static_cast<Tout*>(dinit), part, d, nblk));
  };
  if (K == 2) go(k_conv_bwd<Tin, Tout, V, 2>);
  if (K == 3) go(k_conv_bwd<Tin, Tout, V, 3>);
  if (K == 4) go(k_conv_bwd<Tin, Tout, V, 4>);
  const dim3 rg(ceil_div(d.C, 32), K + 1);
  SSD_LAUNCH("k_conv_dw", s, k_conv_dw<<<rg, 256, 0, s>>>(part, dw, dbias, nparts, d.C, K));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

template <typename Tin, typename Tout, int V>
int launch_step(ConvDims d, int K, const void* x, void* state, const float* w, const float* bias,
                const int* slots, int64_t nslots, void* y, cudaStream_t s) {
  d.nvec = d.C / V;
  const int blocks = ceil_div((int64_t)d.B * d.nvec, 128);
  auto go = [&](auto kern) {
    SSD_LAUNCH("k_conv_step", s,
               kern<<<blocks, 128, 0, s>>>(static_cast<const Tin*>(x), static_cast<Tin*>(state), w,
                                           bias, slots, nslots, static_cast<Tout*>(y), d));
  };
  if (K == 2) go(k_conv_step<Tin, Tout, V, 2>);
  if (K == 3) go(k_conv_step<Tin, Tout, V, 3>);
  if (K == 4) go(k_conv_step<Tin, Tout, V, 4>);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

bool misaligned(const void* p, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(esize - 1)) != 0;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_causal_conv_fwd(const ssd_conv_shape* shape, const void* x, const float* w,
                        const float* bias, const void* init_state, const int32_t* lengths, void* y,
                        void* final_state, void* stream) {
  ConvDims d;
  const int st = conv_dims(shape, &d);
  if (st != SSD_OK) return st;
  if (!x || !w || !y) return SSD_ERR_INVALID_ARG;
  const int K = (int)shape->width;
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4, oe = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (misaligned(x, ie) || misaligned(init_state, ie) || misaligned(final_state, ie) ||
      misaligned(y, oe) || misaligned(w, 4) || misaligned(bias, 4) || misaligned(lengths, 4))
    return SSD_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int v = ie == 2 ? 8 : 4;
  const bool vec = d.C % v == 0 && vec_ok(x, d.xs, ie, v) && vec_ok(x, d.xb, ie, v) && vec_ok(init_state, d.C, ie, v) &&
                   vec_ok(final_state, d.C, ie, v) && vec_ok(y, d.C, oe, v);
#define SSD_GO(TI, TO, V) \
  launch_fwd<TI, TO, V>(d, K, x, w, bias, init_state, lengths, y, final_state, s)
  if (ie == 4) return vec ? SSD_GO(float, float, 4) : SSD_GO(float, float, 1);
  if (oe == 4) return vec ? SSD_GO(bf16, float, 8) : SSD_GO(bf16, float, 1);
  return vec ? SSD_GO(bf16, bf16, 8) : SSD_GO(bf16, bf16, 1);
#undef SSD_GO
}

size_t ssd_causal_conv_workspace_size(const ssd_conv_shape* shape) {
  ConvDims d;
  if (conv_dims(shape, &d) != SSD_OK) return 0;
  d.nvec = ceil_div(d.C, 4);
  bwd_segments(&d);
  return (size_t)bwd_parts(d) * (shape->width + 1) * d.C * sizeof(float);
}

int ssd_causal_conv_bwd(const ssd_conv_shape* shape, const void* x, const float* w,
                        const float* bias, const void* init_state, const int32_t* lengths,
                        const void* dy, const void* dfinal_state, void* dx, float* dw,
                        float* dbias, void* dinit_state, void* workspace, size_t workspace_bytes,
                        void* stream) {
  ConvDims d;
  const int st = conv_dims(shape, &d);
  if (st != SSD_OK) return st;
  if (!x || !w || !dy || !dx || !dw) return SSD_ERR_INVALID_ARG;
  const int K = (int)shape->width;
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4, oe = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (misaligned(x, ie) || misaligned(init_state, ie) || misaligned(dy, ie) ||
      misaligned(dfinal_state, ie) || misaligned(dx, oe) || misaligned(dinit_state, oe) ||
      misaligned(w, 4) || misaligned(bias, 4) || misaligned(dw, 4) || misaligned(dbias, 4) ||
      misaligned(lengths, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, 4) ||
      workspace_bytes < ssd_causal_conv_workspace_size(shape))
    return SSD_ERR_WORKSPACE;
  d.nvec = ceil_div(d.C, 4);
  bwd_segments(&d);
  if (bwd_parts(d) > 65535) return SSD_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  const bool vec = d.C % 4 == 0 && vec_ok(x, d.xs, ie, 4) && vec_ok(x, d.xb, ie, 4) && vec_ok(init_state, d.C, ie, 4) &&
                   vec_ok(dy, d.C, ie, 4) && vec_ok(dfinal_state, d.C, ie, 4) &&
                   vec_ok(dx, d.C, oe, 4) && vec_ok(dinit_state, d.C, oe, 4);
#define SSD_GO(TI, TO, V)                                                                     \
  launch_bwd<TI, TO, V>(d, K, x, w, bias, init_state, lengths, dy, dfinal_state, dx, dw, dbias, \
                        dinit_state, part, s)
  if (ie == 4) return vec ? SSD_GO(float, float, 4) : SSD_GO(float, float, 1);
  if (oe == 4) return vec ? SSD_GO(bf16, float, 4) : SSD_GO(bf16, float, 1);
  return vec ? SSD_GO(bf16, bf16, 4) : SSD_GO(bf16, bf16, 1);
#undef SSD_GO
}

int ssd_causal_conv_step(const ssd_conv_shape* shape, const void* x, void* state, const float* w,
                         const float* bias, const int32_t* slots, int64_t nslots, void* y,
                         void* stream) {
  ConvDims d;
  const int st = conv_dims(shape, &d);
  if (st != SSD_OK) return st;
  if (d.T != 1 || nslots < 1 || (!slots && nslots < d.B)) return SSD_ERR_INVALID_ARG;
  if (!x || !state || !w || !y) return SSD_ERR_INVALID_ARG;
  const int K = (int)shape->width;
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4, oe = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (misaligned(x, ie) || misaligned(state, ie) || misaligned(y, oe) || misaligned(w, 4) ||
      misaligned(bias, 4) || misaligned(slots, 4))
    return SSD_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = d.C % 4 == 0 && vec_ok(x, d.xs, ie, 4) && vec_ok(x, d.xb, ie, 4) && vec_ok(state, d.C, ie, 4) &&
                   vec_ok(y, d.C, oe, 4);
#define SSD_GO(TI, TO, V) \
  launch_step<TI, TO, V>(d, K, x, state, w, bias, slots, nslots, y, s)
  if (ie == 4) return vec ? SSD_GO(float, float, 4) : SSD_GO(float, float, 1);
  if (oe == 4) return vec ? SSD_GO(bf16, float, 4) : SSD_GO(bf16, float, 1);
  return vec ? SSD_GO(bf16, bf16, 4) : SSD_GO(bf16, bf16, 1);
#undef SSD_GO
}

}  // extern "C"
