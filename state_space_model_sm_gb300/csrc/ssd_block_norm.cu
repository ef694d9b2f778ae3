// Block norm: the step between two layers.  With a layer's output o, the
// residual stream r, a residual scale s and an optional gate,
//     t  = o rstd(o) w_post   (or o, without w_post)
//     r' = r + s gate t
//     h  = r' rstd(r') w_pre,     rstd(v) = 1 / sqrt(mean(v^2) + eps)
// so a layer's closing norm, its gate and scale, the residual addition and the
// next layer's opening norm are one pass over r and o.  The backward takes the
// forward's inputs and forms r' again:
//     gx = dh w_pre,  dR = dr' + rstd(r') (gx - xhat mean(gx xhat)),  xhat = r' rstd(r')
//     dr = dR,  dw_pre = sum dh xhat,  dgate = s sum dR t
//     dt = s gate dR,  dw_post = sum dt ohat,  do = rstd(o) (gy - ohat mean(gy ohat)),
//     gy = dt w_post,  ohat = o rstd(o).
// The pages name no kernel for it.
//
// HBM-bound: 12 bytes an element forward and 18 backward (bf16 layer, fp32
// residual) against ~12 and ~30 operations.  A block owns a contiguous range
// of rows and walks it, a thread keeping its columns, so the weight gradients
// stay in registers until the range ends; the row's sums are two (forward) or
// three (backward) block-wide reductions.
#include <cuda_bf16.h>

#include "layer_math.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace lm;
using bf16 = __nv_bfloat16;

struct BnDims {
  int rows, F, ng, gs;  // gs: rows of a gate row
  int R, grid;          // rows of a block; blocks
  float eps, scale;
};

constexpr int kMaxThreads = 512;

// Sums of a and b over the block, in warp order.  Buffers alternate (ph), so one
// barrier a call is enough.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 (*red)[16], int& ph) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) red[ph][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
  for (int i = 0; i < nw; ++i) s.x += red[ph][i].x, s.y += red[ph][i].y;
  ph ^= 1;
  return s;
}

template <typename Tio, typename Tres, int V, int NV>
__global__ void __launch_bounds__(kMaxThreads)
    k_block_norm_fwd(const Tres* __restrict__ r, const Tio* __restrict__ o,
                     const float* __restrict__ w_pre, const float* __restrict__ w_post,
                     const float* __restrict__ gate, Tres* __restrict__ rout, Tio* __restrict__ h,
                     BnDims d) {
  __shared__ float2 red[2][16];
  int ph = 0;
  const float inv = 1.f / (float)d.F;
  const int r0 = blockIdx.x * d.R, r1 = min(d.rows, r0 + d.R);
  for (int row = r0; row < r1; ++row) {
    const int64_t base = (int64_t)row * d.F;
    const float* gp = gate ? gate + (int64_t)(row / d.gs) * d.F : nullptr;
    float ov[NV][V], rv[NV][V], so = 0.f, sr = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * V;
      const bool in = c < d.F;
      unpack<Tio, V>(in ? ld_raw<Tio, V>(o + base + c) : zero_raw<Tio, V>(), ov[v]);
      unpack<Tres, V>(in ? ld_raw<Tres, V>(r + base + c) : zero_raw<Tres, V>(), rv[v]);
#pragma unroll
      for (int i = 0; i < V; ++i) so = fmaf(ov[v][i], ov[v][i], so);
    }
    float ro = 1.f;
    if (w_post) ro = rsqrtf(block_sum2(so, 0.f, red, ph).x * inv + d.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * V;
      if (c >= d.F) continue;
      float wp[V], gt[V];
      if (w_post) unpack<float, V>(ld_raw<float, V>(w_post + c), wp);
      if (gp) unpack<float, V>(ld_raw<float, V>(gp + c), gt);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float t = ov[v][i];
        if (w_post) t *= ro * wp[i];
        if (gp) t *= gt[i];
        rv[v][i] = fmaf(d.scale, t, rv[v][i]);
        sr = fmaf(rv[v][i], rv[v][i], sr);
      }
      st_raw<Tres, V>(rout + base + c, pack<Tres, V>(rv[v]));
    }
    const float rr = rsqrtf(block_sum2(sr, 0.f, red, ph).x * inv + d.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * V;
      if (c >= d.F) continue;
      float wv[V];
      unpack<float, V>(ld_raw<float, V>(w_pre + c), wv);
#pragma unroll
      for (int i = 0; i < V; ++i) rv[v][i] *= rr * wv[i];
      st_raw<Tio, V>(h + base + c, pack<Tio, V>(rv[v]));
    }
  }
}

// part: dw_pre (grid, F), dw_post (grid, F), dgate (grid + ng, F).  A block's
// rows cover the gate rows g of a contiguous range; its part for g is slot
// blockIdx.x + g, which no other (block, gate row) pair has, because from one
// pair that shares rows to the next the block, the gate row or both grow.
template <typename Tio, typename Tres, int V, int NV>
__global__ void __launch_bounds__(kMaxThreads)
    k_block_norm_bwd(const Tres* __restrict__ r, const Tio* __restrict__ o,
                     const float* __restrict__ w_pre, const float* __restrict__ w_post,
                     const float* __restrict__ gate, const Tio* __restrict__ dh,
                     const Tres* __restrict__ drout, Tres* __restrict__ dr, Tio* __restrict__ dout,
                     float* __restrict__ part, BnDims d) {
  __shared__ float2 red[2][16];
  int ph = 0;
  const float inv = 1.f / (float)d.F;
  const int r0 = blockIdx.x * d.R, r1 = min(d.rows, r0 + d.R);
  float apre[NV][V], apost[NV][V], agate[NV][V];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < V; ++i) apre[v][i] = apost[v][i] = agate[v][i] = 0.f;
  float* const pgate = part + 2 * (int64_t)d.grid * d.F;
  for (int row = r0; row < r1; ++row) {
    const int64_t base = (int64_t)row * d.F;
    const float* gp = gate ? gate + (int64_t)(row / d.gs) * d.F : nullptr;
    float ov[NV][V], rv[NV][V], hv[NV][V], so = 0.f, sr = 0.f, sx = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * V;
      const bool in = c < d.F;
      unpack<Tio, V>(in ? ld_raw<Tio, V>(o + base + c) : zero_raw<Tio, V>(), ov[v]);
      unpack<Tres, V>(in ? ld_raw<Tres, V>(r + base + c) : zero_raw<Tres, V>(), rv[v]);
      unpack<Tio, V>(in ? ld_raw<Tio, V>(dh + base + c) : zero_raw<Tio, V>(), hv[v]);
#pragma unroll
      for (int i = 0; i < V; ++i) so = fmaf(ov[v][i], ov[v][i], so);
    }
    float ro = 1.f;
    if (w_post) ro = rsqrtf(block_sum2(so, 0.f, red, ph).x * inv + d.eps);
    // ov: ohat; rv: r'
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * V;
      if (c >= d.F) continue;
      float wp[V], gt[V], wv[V];
      if (w_post) unpack<float, V>(ld_raw<float, V>(w_post + c), wp);
      if (gp) unpack<float, V>(ld_raw<float, V>(gp + c), gt);
      unpack<float, V>(ld_raw<float, V>(w_pre + c), wv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ov[v][i] *= ro;
        float t = ov[v][i];
        if (w_post) t *= wp[i];
        if (gp) t *= gt[i];
        rv[v][i] = fmaf(d.scale, t, rv[v][i]);
        sr = fmaf(rv[v][i], rv[v][i], sr);
        sx = fmaf(hv[v][i] * wv[i], rv[v][i], sx);
      }
    }
    const float2 s2 = block_sum2(sr, sx, red, ph);
    const float rr = rsqrtf(s2.x * inv + d.eps), cx = s2.y * inv * rr * rr;
    float sy = 0.f;
    // rv: dR; hv: dt
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * V;
      if (c >= d.F) continue;
      float wp[V], gt[V], wv[V], dv[V];
      if (w_post) unpack<float, V>(ld_raw<float, V>(w_post + c), wp);
      if (gp) unpack<float, V>(ld_raw<float, V>(gp + c), gt);
      unpack<float, V>(ld_raw<float, V>(w_pre + c), wv);
      unpack<Tres, V>(drout ? ld_raw<Tres, V>(drout + base + c) : zero_raw<Tres, V>(), dv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        apre[v][i] = fmaf(hv[v][i], rv[v][i] * rr, apre[v][i]);
        rv[v][i] = dv[i] + rr * (hv[v][i] * wv[i] - rv[v][i] * cx);
        float dt = d.scale * rv[v][i];
        if (gp) {
          agate[v][i] = fmaf(dt, w_post ? ov[v][i] * wp[i] : ov[v][i], agate[v][i]);
          dt *= gt[i];
        }
        if (w_post) {
          apost[v][i] = fmaf(dt, ov[v][i], apost[v][i]);
          dt *= wp[i];
        }
        hv[v][i] = dt;
        sy = fmaf(dt, ov[v][i], sy);
      }
      st_raw<Tres, V>(dr + base + c, pack<Tres, V>(rv[v]));
    }
    float cy = 0.f;
    if (w_post) cy = block_sum2(sy, 0.f, red, ph).x * inv;
    const bool flush = gp && (row + 1 == r1 || (row + 1) % d.gs == 0);
    float* pg = pgate + (int64_t)(blockIdx.x + row / d.gs) * d.F;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * V;
      if (c >= d.F) continue;
      if (w_post) {
#pragma unroll
        for (int i = 0; i < V; ++i) hv[v][i] = ro * (hv[v][i] - ov[v][i] * cy);
      }
      st_raw<Tio, V>(dout + base + c, pack<Tio, V>(hv[v]));
      if (flush) {
        st_raw<float, V>(pg + c, pack<float, V>(agate[v]));
#pragma unroll
        for (int i = 0; i < V; ++i) agate[v][i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * V;
    if (c >= d.F) continue;
    st_raw<float, V>(part + (int64_t)blockIdx.x * d.F + c, pack<float, V>(apre[v]));
    if (w_post)
      st_raw<float, V>(part + (int64_t)(d.grid + blockIdx.x) * d.F + c, pack<float, V>(apost[v]));
  }
}

// dw_pre, dw_post and the gate rows' gradients: the blocks' parts in a fixed
// order, 32 columns a block, its 8 warps taking every 8th part.
// blockIdx.y = 0: dw_pre, 1: dw_post, 2 + g: gate row g.
__global__ void __launch_bounds__(256)
    k_block_norm_dw(const float* __restrict__ part, float* __restrict__ dw_pre,
                    float* __restrict__ dw_post, float* __restrict__ dgate, BnDims d) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, which = blockIdx.y, g = which - 2;
  int k0 = 0, k1 = d.grid;
  const float* p = part + (which == 1 ? (int64_t)d.grid * d.F : 0);
  float* dst = which == 0 ? dw_pre : dw_post;
  if (which >= 2) {
    k0 = (int)((int64_t)g * d.gs / d.R);
    k1 = (int)((((int64_t)g + 1) * d.gs - 1) / d.R) + 1;
    p = part + (2 * (int64_t)d.grid + g) * d.F;
    dst = dgate + (int64_t)g * d.F;
  }
  if (!dst) return;
  float a = 0.f;
  if (c < d.F)
    for (int k = k0 + warp; k < k1; k += 8) a += p[(int64_t)k * d.F + c];
  red[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < d.F) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][lane];
    dst[c] = s;
  }
}

// ------------------------------------------------------------------- host

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int bn_dims(const ssd_block_norm_shape* s, BnDims* d) {
  if (!s || s->rows < 0 || s->features < 1 || s->ngates < 0 || !(s->eps >= 0.f) ||
      !(s->scale == s->scale))
    return SSD_ERR_INVALID_ARG;
  if ((s->in_dtype != SSD_F32 && s->in_dtype != SSD_BF16) ||
      (s->res_dtype != SSD_F32 && s->res_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  if (s->rows >= (1 << 30) || (s->ngates && s->rows % s->ngates != 0)) return SSD_ERR_INVALID_ARG;
  if (s->features > 8192) return SSD_ERR_UNSUPPORTED;
  if (s->in_dtype == SSD_F32 && s->res_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  d->rows = (int)s->rows, d->F = (int)s->features, d->ng = (int)s->ngates;
  d->gs = d->ng && d->rows ? d->rows / d->ng : (d->rows ? d->rows : 1);
  d->eps = s->eps, d->scale = s->scale;
  return SSD_OK;
}

// Row ranges: as many blocks as are resident at once (1024 threads an SM),
// each with the same number of consecutive rows.
void bn_grid(BnDims* d) {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms = 152;
  const int nt = d->F >= 4096 ? 512 : d->F >= 2048 ? 256 : 128;  // threads, about
  d->R = ceil_div(d->rows, (int64_t)sms * (1024 / nt));
  d->grid = ceil_div(d->rows, d->R);
}

size_t bn_part_floats(const BnDims& d) { return ((size_t)3 * d.grid + d.ng) * d.F; }

struct BnPtrs {
  const void *r, *o;
  const float *w_pre, *w_post, *gate;
  const void *dh, *drout;
  void *rout, *h;  // forward outputs; the backward's dr and do
  float* part;
};

template <typename Tio, typename Tres, int V, int NV>
int bn_launch(const BnDims& d, const BnPtrs& p, bool bwd, cudaStream_t s) {
  const int nt = ceil_div(ceil_div(d.F, V * NV), 32) * 32;
  const Tres* r = static_cast<const Tres*>(p.r);
  const Tio* o = static_cast<const Tio*>(p.o);
  if (bwd)
    SSD_LAUNCH("k_block_norm_bwd", s,
               k_block_norm_bwd<Tio, Tres, V, NV><<<d.grid, nt, 0, s>>>(
                   r, o, p.w_pre, p.w_post, p.gate, static_cast<const Tio*>(p.dh),
                   static_cast<const Tres*>(p.drout), static_cast<Tres*>(p.rout),
                   static_cast<Tio*>(p.h), p.part, d));
  else
    SSD_LAUNCH("k_block_norm_fwd", s,
               k_block_norm_fwd<Tio, Tres, V, NV><<<d.grid, nt, 0, s>>>(
                   r, o, p.w_pre, p.w_post, p.gate, static_cast<Tres*>(p.rout),
                   static_cast<Tio*>(p.h), d));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// 8 columns a thread (one 16-byte access of bf16, two of fp32) where rows
// divide into them, else single columns; then twice as many per thread until a
// row fits 512 threads.
template <typename Tio, typename Tres>
int bn_pick(const BnDims& d, const BnPtrs& p, bool vec, bool bwd, cudaStream_t s) {
  if (vec) {
    if (d.F <= 8 * kMaxThreads) return bn_launch<Tio, Tres, 8, 1>(d, p, bwd, s);
    return bn_launch<Tio, Tres, 8, 2>(d, p, bwd, s);
  }
  if (d.F <= kMaxThreads) return bn_launch<Tio, Tres, 1, 1>(d, p, bwd, s);
  if (d.F <= 4 * kMaxThreads) return bn_launch<Tio, Tres, 1, 4>(d, p, bwd, s);
  return bn_launch<Tio, Tres, 1, 16>(d, p, bwd, s);
}

int bn_run(const BnDims& d, const ssd_block_norm_shape* sh, const BnPtrs& p, bool vec, bool bwd,
           cudaStream_t s) {
  if (sh->in_dtype == SSD_F32) return bn_pick<float, float>(d, p, vec, bwd, s);
  if (sh->res_dtype == SSD_F32) return bn_pick<bf16, float>(d, p, vec, bwd, s);
  return bn_pick<bf16, bf16>(d, p, vec, bwd, s);
}

bool off(const void* p, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(esize - 1)) != 0;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_block_norm_workspace_size(const ssd_block_norm_shape* shape) {
  BnDims d;
  if (bn_dims(shape, &d) != SSD_OK) return 0;
  if (d.rows == 0) return 256;
  bn_grid(&d);
  return bn_part_floats(d) * sizeof(float);
}

int ssd_block_norm_fwd(const ssd_block_norm_shape* shape, const void* residual, const void* o,
                       const float* w_pre, const float* w_post, const float* gate,
                       void* residual_out, void* h, void* stream) {
  BnDims d;
  const int st = bn_dims(shape, &d);
  if (st != SSD_OK) return st;
  if (d.rows == 0) return SSD_OK;
  if (!residual || !o || !w_pre || !residual_out || !h || (d.ng != 0) != (gate != nullptr))
    return SSD_ERR_INVALID_ARG;
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4, re = shape->res_dtype == SSD_BF16 ? 2 : 4;
  if (off(residual, re) || off(residual_out, re) || off(o, ie) || off(h, ie) || off(w_pre, 4) ||
      off(w_post, 4) || off(gate, 4))
    return SSD_ERR_INVALID_ARG;
  bn_grid(&d);
  const bool vec = vec_ok(o, d.F, ie, 8) && vec_ok(h, d.F, ie, 8) && vec_ok(residual, d.F, re, 8) &&
                   vec_ok(residual_out, d.F, re, 8) && vec_ok(w_pre, d.F, 4, 8) &&
                   vec_ok(w_post, d.F, 4, 8) && vec_ok(gate, d.F, 4, 8) && d.F % 8 == 0;
  const BnPtrs p{residual, o, w_pre, w_post, gate, nullptr, nullptr, residual_out, h, nullptr};
  return bn_run(d, shape, p, vec, false, static_cast<cudaStream_t>(stream));
}

int ssd_block_norm_bwd(const ssd_block_norm_shape* shape, const void* residual, const void* o,
                       const float* w_pre, const float* w_post, const float* gate, const void* dh,
                       const void* dresidual_out, void* dresidual, void* d_o, float* dw_pre,
                       float* dw_post, float* dgate, void* workspace, size_t workspace_bytes,
                       void* stream) {
  BnDims d;
  const int st = bn_dims(shape, &d);
  if (st != SSD_OK) return st;
  if (!w_pre || !dw_pre || (w_post != nullptr) != (dw_post != nullptr) ||
      (d.ng != 0) != (gate != nullptr) || (gate != nullptr) != (dgate != nullptr))
    return SSD_ERR_INVALID_ARG;
  if (d.rows > 0 && (!residual || !o || !dh || !dresidual || !d_o)) return SSD_ERR_INVALID_ARG;
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4, re = shape->res_dtype == SSD_BF16 ? 2 : 4;
  if (off(residual, re) || off(dresidual_out, re) || off(dresidual, re) || off(o, ie) ||
      off(dh, ie) || off(d_o, ie) || off(w_pre, 4) || off(w_post, 4) || off(gate, 4) ||
      off(dw_pre, 4) || off(dw_post, 4) || off(dgate, 4))
    return SSD_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d.rows == 0) {  // no rows: the weight gradients are 0
    const size_t n = (size_t)d.F * sizeof(float);
    bool ok = cudaMemsetAsync(dw_pre, 0, n, s) == cudaSuccess;
    if (dw_post) ok = ok && cudaMemsetAsync(dw_post, 0, n, s) == cudaSuccess;
    if (dgate) ok = ok && cudaMemsetAsync(dgate, 0, n * d.ng, s) == cudaSuccess;
    return ok ? SSD_OK : SSD_ERR_CUDA;
  }
  bn_grid(&d);
  if (!workspace || off(workspace, 16) || workspace_bytes < bn_part_floats(d) * sizeof(float))
    return SSD_ERR_WORKSPACE;
  if (d.ng + 2 > 65535) return SSD_ERR_UNSUPPORTED;
  const bool vec = d.F % 8 == 0 && vec_ok(o, d.F, ie, 8) && vec_ok(dh, d.F, ie, 8) &&
                   vec_ok(d_o, d.F, ie, 8) && vec_ok(residual, d.F, re, 8) &&
                   vec_ok(dresidual_out, d.F, re, 8) && vec_ok(dresidual, d.F, re, 8) &&
                   vec_ok(w_pre, d.F, 4, 8) && vec_ok(w_post, d.F, 4, 8) && vec_ok(gate, d.F, 4, 8);
  const BnPtrs p{residual, o, w_pre, w_post, gate, dh, dresidual_out, dresidual, d_o,
                 static_cast<float*>(workspace)};
  const int e = bn_run(d, shape, p, vec, true, s);
  if (e != SSD_OK) return e;
  const dim3 grid(ceil_div(d.F, 32), 2 + d.ng);
  SSD_LAUNCH("k_block_norm_dw", s,
             k_block_norm_dw<<<grid, 256, 0, s>>>(p.part, dw_pre, dw_post, dgate, d));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
