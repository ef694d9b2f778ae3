// Block norm: the step between two layers.  With a layer's output o, the
// residual stream r, a residual scale s and an optional gate,
//     t  = o rstd(o) w_post   (or o, without w_post)
//     r' = r + s gate t
//     h  = r' rstd(r') w_pre,     rstd(v) = 1 / sqrt(mean(v^2) + eps)
// so a layer's closing norm, its gate and scale, the residual addition and the
// next layer's opening norm are one pass over r and o.  The backward takes the
// forward's inputs and forms r' again:
//     gx = dh w_pre,  dR = dr' + rstd(r') (gx - xhat mean(gx xhat)),  xhat = r' rstd(r')
//     dr = dR,  dw_pre = sum dh xhat,  do = rstd(o) (gy - ohat mean(gy ohat)),
//     gy = s gate w_post dR,  ohat = o rstd(o)
// and, with P_g = sum of dR ohat over the rows of gate row g,
//     dgate_g = s w_post P_g,  dw_post = sum_g s gate_g P_g,
// so two sums over rows give all three gradients.
//
// HBM-bound: 12 bytes an element forward and 18 backward (bf16 layer, fp32
// residual).  At 16384 x 4096 it takes 133 and 196 us (6.1 and 6.2 TB/s, 0.90 of a
// plain copy's rate) with 33 and 41 % of the issue slots, so the arithmetic has to
// be lean: it is in packed pairs, an absent weight or gate is a vector of ones (no
// branches), and a thread owns 16 columns, over which the two (forward) or three
// (backward) block-wide sums of a row are spread; their barriers are the first
// stall of the backward.  bf16 residuals halve the bytes but not the sums: 0.73
// at 8192 columns, 0.80 at 2048; rows of an odd number of bf16 columns, which are
// read one by one, 0.33 to 0.40.  A few rows are bound by their launches.  A block owns a
// contiguous range of rows and walks it, a thread keeping its columns, so the
// weight gradients stay in registers until the range ends.
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
  int nt, S;            // threads of a block; ring stages
  float eps, scale;
};

constexpr int kMaxThreads = 512;
constexpr int kMaxStages = 4;

// Sums over the block of v (both components), in warp order.  Buffers alternate
// (ph), so one barrier a call is enough.
__device__ __forceinline__ float2 block_sum(float2 v, float2 (*red)[16], int& ph) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                            __shfl_xor_sync(0xffffffffu, v.y, o)));
  const int nw = blockDim.x >> 5, pw = nw > 8 ? 16 : nw > 4 ? 8 : nw > 2 ? 4 : 2;
  const int i = threadIdx.x & (pw - 1);  // every aligned group of pw lanes adds the warps' sums
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) red[ph][threadIdx.x >> 5] = v;
  __syncthreads();
  v = i < nw ? red[ph][i] : f2(0.f);
  for (int o = pw / 2; o > 0; o >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                            __shfl_xor_sync(0xffffffffu, v.y, o)));
  ph ^= 1;
  return v;
}
__device__ __forceinline__ float block_sum(float a, float2 (*red)[16], int& ph) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  const int nw = blockDim.x >> 5, pw = nw > 8 ? 16 : nw > 4 ? 8 : nw > 2 ? 4 : 2;
  const int i = threadIdx.x & (pw - 1);  // every aligned group of pw lanes adds the warps' sums
  if (nw == 1) return a;
  if ((threadIdx.x & 31) == 0) red[ph][threadIdx.x >> 5].x = a;
  __syncthreads();
  a = i < nw ? red[ph][i].x : 0.f;
  for (int o = pw / 2; o > 0; o >>= 1)
    a += __shfl_xor_sync(0xffffffffu, a, o);
  ph ^= 1;
  return a;
}

// A thread's EPT columns, as pairs, in pieces of VEC consecutive columns, the
// threads' pieces side by side, so every access of a warp is one unbroken run.
// VEC is 8 where layer and residual are bf16 (16-byte pieces: 88 us at 16384 x
// 1000 forward and backward and 270 at 8192 x 8192, against 108 and 290 with 4);
// 4 where one of them is fp32 (16 bytes; 8 would be 32-byte pieces, whose 16-byte
// halves touch each sector twice: 20 % slower), or where the width or an address
// fits only 4; 0 where none fits: single columns, blockDim.x apart.
// FULL: the row is exactly the block's columns (no bounds to check).
template <int VEC, int EPT, bool FULL>
struct Cols {
  static constexpr int W = VEC ? VEC : 1, P2 = EPT / 2, NV = EPT / W;
  __device__ __forceinline__ static int col(int v) {
    return (v * (int)blockDim.x + (int)threadIdx.x) * W;
  }
  template <typename T>
  __device__ __forceinline__ static void load(const T* p, int F, float2 (&x)[P2], float fill) {
    float* f = reinterpret_cast<float*>(x);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = col(v);
      float t[W];
      if ((FULL || c < F) && p) {
        unpack<T, W>(ld_raw<T, W>(p + c), t);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) t[i] = fill;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) f[v * W + i] = t[i];
    }
  }
  template <typename T>
  __device__ __forceinline__ static void store(T* p, int F, const float2 (&x)[P2]) {
    const float* f = reinterpret_cast<const float*>(x);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = col(v);
      if (!FULL && c >= F) break;
      float t[W];
#pragma unroll
      for (int i = 0; i < W; ++i) t[i] = f[v * W + i];
      st_raw<T, W>(p + c, pack<T, W>(t));
    }
  }
};

// A block's rows of its inputs.  VEC != 0: a ring in shared memory; a thread copies the
// pieces that it will use itself, S - 1 rows ahead, so the bytes in flight are
// set by the ring and no barrier is needed.  Else plain loads of the row.
// Addresses advance by a row at a time.
template <typename Tio, typename Tres, int VEC, int EPT, bool FULL, int NIO, int NRES>
struct Rows {
  using C = Cols<VEC, EPT, FULL>;
  static constexpr int NV = VEC ? C::NV : 0;
  // bytes of a thread's piece of one tensor, of its row of one, of its slot
  static constexpr int kIo = VEC * sizeof(Tio), kRes = VEC * sizeof(Tres);
  static constexpr int kSlot = NV * (NIO * kIo + NRES * kRes);
  const Tio* io[NIO];     // VEC: this thread's first column of the next row to copy;
  const Tres* res[NRES];  // else the row in use
  // single columns, 8 a thread: the next row in registers (more would not fit)
  static constexpr bool kReg = !VEC && EPT <= 8;
  static constexpr int NR = kReg ? EPT : 1;
  Tio cio[NIO][NR], nio[NIO][NR];
  Tres cres[NRES][NR], nres[NRES][NR];
  uint32_t put, use, end, slot;  // ring offsets: next copy's slot, the row in use; end; a slot
  uint32_t iostep, resstep;      // bytes of the block's pieces v of one tensor
  int F, S, left, pieces;        // left: rows still to copy; pieces: of this thread in a row

  __device__ __forceinline__ static unsigned char* smem() {
    extern __shared__ __align__(16) unsigned char ring[];
    return ring;
  }
  __device__ __forceinline__ void start(int width, int stages, int r0, int r1) {
    F = width, S = stages, left = r1 - r0;
    const int64_t at = VEC ? (int64_t)r0 * F + C::col(0) : ((int64_t)r0 - (kReg ? 0 : 1)) * F;
#pragma unroll
    for (int i = 0; i < NIO; ++i) io[i] += at;
#pragma unroll
    for (int i = 0; i < NRES; ++i)
      if (res[i]) res[i] += at;
    if constexpr (VEC) {
      iostep = kIo * blockDim.x, resstep = kRes * blockDim.x;
      pieces = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) pieces += C::col(v) < F;
      slot = kSlot * blockDim.x, end = S * slot, put = 0, use = end - slot;
      for (int i = 0; i < S - 1; ++i) fill();
    } else if constexpr (kReg) {
      fetch();
    }
  }
  __device__ __forceinline__ void fetch() {  // the next row into registers
    if (left > 0) {
#pragma unroll
      for (int v = 0; v < NR; ++v) {
        const int c = C::col(v);
#pragma unroll
        for (int i = 0; i < NIO; ++i) nio[i][v] = c < F ? io[i][c] : from_f<Tio>(0.f);
#pragma unroll
        for (int i = 0; i < NRES; ++i)
          nres[i][v] = c < F && res[i] ? res[i][c] : from_f<Tres>(0.f);
      }
      advance();
      --left;
    }
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int i = 0; i < NIO; ++i) io[i] += F;
#pragma unroll
    for (int i = 0; i < NRES; ++i)
      if (res[i]) res[i] += F;
  }
  // offset in a slot of this thread's first piece of tensor i (io first, then res)
  __device__ __forceinline__ uint32_t io_at(int i) const {
    return i * NV * iostep + threadIdx.x * kIo;
  }
  __device__ __forceinline__ uint32_t res_at(int i) const {
    return NIO * NV * iostep + i * NV * resstep + threadIdx.x * kRes;
  }
  __device__ __forceinline__ void fill() {  // the next row, into the next slot
    if (left > 0) {
      unsigned char* const q = smem() + put;
      const int cols = VEC * blockDim.x;
#pragma unroll
      for (int i = 0; i < NIO; ++i)
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (FULL || v < pieces) cp_async<kIo>(q + io_at(i) + v * iostep, io[i] + v * cols);
#pragma unroll
      for (int i = 0; i < NRES; ++i)
        if (res[i]) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
            if (FULL || v < pieces) cp_async<kRes>(q + res_at(i) + v * resstep, res[i] + v * cols);
        }
      advance();
      --left;
      put = put + slot == end ? 0 : put + slot;
    }
    cp_commit();
  }
  // Makes the next row readable and starts the copy of the one S - 1 further,
  // into the slot that this thread read last.
  __device__ __forceinline__ void next() {
    if constexpr (VEC) {
      use = use + slot == end ? 0 : use + slot;
      if (S == 1) {  // no room for a second row: copied when it is needed
        fill();
        cp_wait<0>();
        return;
      }
      if (S == 4)
        cp_wait<2>();
      else if (S == 3)
        cp_wait<1>();
      else
        cp_wait<0>();
      fill();
    } else if constexpr (kReg) {
#pragma unroll
      for (int v = 0; v < NR; ++v) {
#pragma unroll
        for (int i = 0; i < NIO; ++i) cio[i][v] = nio[i][v];
#pragma unroll
        for (int i = 0; i < NRES; ++i) cres[i][v] = nres[i][v];
      }
      fetch();
    } else {
      advance();
    }
  }
  __device__ __forceinline__ void get_io(int i, float2 (&x)[C::P2]) const {
    if constexpr (VEC)
      get<Tio>(io_at(i), iostep, pieces, x);
    else if constexpr (kReg)
      of_regs(cio[i], x);
    else
      C::load(io[i], F, x, 0.f);
  }
  __device__ __forceinline__ void get_res(int i, float2 (&x)[C::P2]) const {
    if constexpr (VEC) {
      if (res[i]) {
        get<Tres>(res_at(i), resstep, pieces, x);
      } else {
#pragma unroll
        for (int k = 0; k < C::P2; ++k) x[k] = f2(0.f);
      }
    } else if constexpr (kReg) {
      of_regs(cres[i], x);
    } else {
      C::load(res[i], F, x, 0.f);
    }
  }
  template <typename T>
  __device__ __forceinline__ static void of_regs(const T (&r)[NR], float2 (&x)[C::P2]) {
#pragma unroll
    for (int k = 0; k < C::P2; ++k) x[k] = make_float2(to_f(r[2 * k]), to_f(r[2 * k + 1]));
  }
  template <typename T>
  __device__ __forceinline__ void get(uint32_t at, uint32_t step, int n, float2 (&x)[C::P2]) const {
    float* f = reinterpret_cast<float*>(x);
    const unsigned char* q = smem() + use + at;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Raw<T, C::W> r = zero_raw<T, C::W>();
      if (FULL || v < n) r = *reinterpret_cast<const Raw<T, C::W>*>(q + v * step);
      float t[C::W];
      unpack<T, C::W>(r, t);
#pragma unroll
      for (int k = 0; k < C::W; ++k) f[v * C::W + k] = t[k];
    }
  }
};

// d r' / d ohat of a thread's columns: s gate_g w_post (absent vectors: ones).
template <typename C>
__device__ __forceinline__ void load_gw(float2 (&gw)[C::P2], const float* w_post, const float* gate,
                                        int g, const BnDims& d) {
  float2 t[C::P2];
  C::load(w_post, d.F, gw, 1.f);
  C::load(gate ? gate + (int64_t)g * d.F : gate, d.F, t, 1.f);
#pragma unroll
  for (int i = 0; i < C::P2; ++i) gw[i] = mul2(gw[i], mul2(t[i], f2(d.scale)));
}

// rout may be r and h may be o: a thread reads its columns of a row before it writes
// them, and nothing else does either, so these four are not __restrict__.
template <typename Tio, typename Tres, int VEC, int EPT, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, 1)
    k_block_norm_fwd(const Tres* r, const Tio* o, const float* __restrict__ w_pre,
                     const float* __restrict__ w_post, const float* __restrict__ gate, Tres* rout,
                     Tio* h, BnDims d) {
  using C = Cols<VEC, EPT, FULL>;
  constexpr int P2 = C::P2;
  __shared__ float2 red[2][16];
  int ph = 0;
  const float inv = 1.f / (float)d.F;
  const int r0 = blockIdx.x * d.R, r1 = min(d.rows, r0 + d.R);
  Rows<Tio, Tres, VEC, EPT, FULL, 1, 1> in;
  in.io[0] = o, in.res[0] = r;
  in.start(d.F, d.S, r0, r1);
  float2 gw[P2], wp[P2];
  C::load(w_pre, d.F, wp, 0.f);
  int g = r0 / d.gs, gend = (g + 1) * d.gs;  // the gate row in use, and where it ends
  load_gw<C>(gw, w_post, gate, g, d);
  rout += (int64_t)r0 * d.F;
  h += (int64_t)r0 * d.F;
  for (int row = r0; row < r1; ++row, rout += d.F, h += d.F) {
    if (row == gend) {
      load_gw<C>(gw, w_post, gate, ++g, d);
      gend += d.gs;
    }
    in.next();
    float2 ov[P2], rv[P2];
    in.get_io(0, ov);
    float ro = 1.f;
    if (w_post) {
      float2 so = f2(0.f);
#pragma unroll
      for (int i = 0; i < P2; ++i) so = fma2(ov[i], ov[i], so);
      ro = rsqrtf(block_sum(so.x + so.y, red, ph) * inv + d.eps);
    }
    in.get_res(0, rv);
    float2 sr = f2(0.f);
#pragma unroll
    for (int i = 0; i < P2; ++i) {
      rv[i] = fma2(mul2(ov[i], f2(ro)), gw[i], rv[i]);
      sr = fma2(rv[i], rv[i], sr);
    }
    C::store(rout, d.F, rv);
    const float rr = rsqrtf(block_sum(sr.x + sr.y, red, ph) * inv + d.eps);
#pragma unroll
    for (int i = 0; i < P2; ++i) rv[i] = mul2(mul2(rv[i], f2(rr)), wp[i]);
    C::store(h, d.F, rv);
  }
}

// part: dw_pre (grid, F), P (grid + gate rows, F).  A block's rows cover the gate
// rows g of a contiguous range (all rows are one without a gate); its part of
// P_g is slot blockIdx.x + g, which no other (block, gate row) pair has, because
// from one pair that shares rows to the next the block, the gate row or both
// grow.
template <typename Tio, typename Tres, int VEC, int EPT, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, 1)
    k_block_norm_bwd(const Tres* __restrict__ r, const Tio* __restrict__ o,
                     const float* __restrict__ w_pre, const float* __restrict__ w_post,
                     const float* __restrict__ gate, const Tio* __restrict__ dh,
                     const Tres* __restrict__ drout, Tres* __restrict__ dr, Tio* __restrict__ dout,
                     float* __restrict__ part, BnDims d) {
  using C = Cols<VEC, EPT, FULL>;
  constexpr int P2 = C::P2;
  __shared__ float2 red[2][16];
  griddep_launch_dependents();
  int ph = 0;
  const float inv = 1.f / (float)d.F;
  const int r0 = blockIdx.x * d.R, r1 = min(d.rows, r0 + d.R);
  Rows<Tio, Tres, VEC, EPT, FULL, 2, 2> in;
  in.io[0] = o, in.io[1] = dh, in.res[0] = r, in.res[1] = drout;
  in.start(d.F, d.S, r0, r1);
  float2 apre[P2], ap[P2], gw[P2], wp[P2];
  C::load(w_pre, d.F, wp, 0.f);
#pragma unroll
  for (int i = 0; i < P2; ++i) apre[i] = ap[i] = f2(0.f);
  float* const pp = part + (int64_t)d.grid * d.F;
  int g = r0 / d.gs, gend = (g + 1) * d.gs;  // the gate row in use, and where it ends
  load_gw<C>(gw, w_post, gate, g, d);
  dr += (int64_t)r0 * d.F;
  dout += (int64_t)r0 * d.F;
  for (int row = r0; row < r1; ++row, dr += d.F, dout += d.F) {
    in.next();
    float2 ov[P2], rv[P2], t[P2];
    in.get_io(0, ov);
    float ro = 1.f;
    if (w_post) {
      float2 so = f2(0.f);
#pragma unroll
      for (int i = 0; i < P2; ++i) so = fma2(ov[i], ov[i], so);
      ro = rsqrtf(block_sum(so.x + so.y, red, ph) * inv + d.eps);
#pragma unroll
      for (int i = 0; i < P2; ++i) ov[i] = mul2(ov[i], f2(ro));  // ohat
    }
    in.get_res(0, rv);
    in.get_io(1, t);  // dh
    float2 sr = f2(0.f), sx = f2(0.f);
#pragma unroll
    for (int i = 0; i < P2; ++i) {
      rv[i] = fma2(gw[i], ov[i], rv[i]);  // r'
      sr = fma2(rv[i], rv[i], sr);
      sx = fma2(mul2(t[i], wp[i]), rv[i], sx);
    }
    const float2 s2 = block_sum(make_float2(sr.x + sr.y, sx.x + sx.y), red, ph);
    const float rr = rsqrtf(s2.x * inv + d.eps), cx = s2.y * inv * rr * rr;
#pragma unroll
    for (int i = 0; i < P2; ++i) {
      apre[i] = fma2(t[i], mul2(rv[i], f2(rr)), apre[i]);
      rv[i] = fma2(t[i], wp[i], mul2(rv[i], f2(-cx)));
    }
    in.get_res(1, t);  // dr'
    float2 sy = f2(0.f);
#pragma unroll
    for (int i = 0; i < P2; ++i) {
      rv[i] = fma2(rv[i], f2(rr), t[i]);  // dR
      ap[i] = fma2(rv[i], ov[i], ap[i]);
    }
    C::store(dr, d.F, rv);
#pragma unroll
    for (int i = 0; i < P2; ++i) {
      rv[i] = mul2(rv[i], gw[i]);  // gy
      sy = fma2(rv[i], ov[i], sy);
    }
    if (w_post) {
      const float cy = block_sum(sy.x + sy.y, red, ph) * inv;
#pragma unroll
      for (int i = 0; i < P2; ++i) rv[i] = mul2(fma2(ov[i], f2(-cy), rv[i]), f2(ro));
    }
    C::store(dout, d.F, rv);
    if (row + 1 == gend || row + 1 == r1) {  // the gate row's part ends
      C::store(pp + (int64_t)(blockIdx.x + g) * d.F, d.F, ap);
      if (row + 1 < r1) {
#pragma unroll
        for (int i = 0; i < P2; ++i) ap[i] = f2(0.f);
        load_gw<C>(gw, w_post, gate, ++g, d);
        gend += d.gs;
      }
    }
  }
  C::store(part + (int64_t)blockIdx.x * d.F, d.F, apre);
}

// dw_pre, dw_post and the gate rows' gradients from the blocks' parts in a fixed
// order, 32 columns a block, its 16 warps taking every 16th block's part.
// Results: 0 is dw_pre, 1 dw_post, 2 + g gate row g.  blockIdx.y is a block's first;
// where there are more than a grid has rows of blocks, it goes on a grid further.
constexpr int kMaxGridY = 65535;

__global__ void __launch_bounds__(512)
    k_block_norm_dw(const float* __restrict__ part, const float* __restrict__ w_post,
                    const float* __restrict__ gate, float* __restrict__ dw_pre,
                    float* __restrict__ dw_post, float* __restrict__ dgate, BnDims d) {
  __shared__ float red[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  griddep_wait();
  const float* pp = part + (int64_t)d.grid * d.F;
  for (int which = blockIdx.y; which < 2 + d.ng; which += gridDim.y) {
    const int g = which - 2;
    float* const dst = which == 0 ? dw_pre : which == 1 ? dw_post : dgate + (int64_t)g * d.F;
    if (!dst) continue;  // no dw_post
    float a = 0.f;
    if (c < d.F) {
      if (which == 0) {
#pragma unroll 8
        for (int k = warp; k < d.grid; k += 16) a += part[(int64_t)k * d.F + c];
      } else if (which == 1 && d.ng <= 16) {  // gate row by gate row
        for (int i = 0; i < (d.ng ? d.ng : 1); ++i) {
          const int k0 = i * d.gs / d.R, k1 = ((i + 1) * d.gs - 1) / d.R + 1;
          float p = 0.f;
#pragma unroll 8
          for (int k = k0 + warp; k < k1; k += 16) p += pp[(int64_t)(k + i) * d.F + c];
          a = fmaf(gate ? gate[(int64_t)i * d.F + c] : 1.f, p, a);
        }
      } else if (which == 1) {  // block by block
        for (int k = warp; k < d.grid; k += 16) {
          const int g0 = k * d.R / d.gs, g1 = (min((k + 1) * d.R, d.rows) - 1) / d.gs;
          for (int i = g0; i <= g1; ++i)
            a = fmaf(gate[(int64_t)i * d.F + c], pp[(int64_t)(k + i) * d.F + c], a);
        }
      } else {
        const int k0 = (int)((int64_t)g * d.gs / d.R);
        const int k1 = (int)((((int64_t)g + 1) * d.gs - 1) / d.R) + 1;
#pragma unroll 8
        for (int k = k0 + warp; k < k1; k += 16) a += pp[(int64_t)(k + g) * d.F + c];
      }
    }
    red[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < d.F) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) s += red[k][lane];
      dst[c] = which == 0 ? s : d.scale * (which == 1 || !w_post ? s : w_post[c] * s);
    }
    if (which + (int64_t)gridDim.y < 2 + d.ng) __syncthreads();  // before the sums' next use
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
  if (s->ngates && s->rows % s->ngates != 0) return SSD_ERR_INVALID_ARG;
  if (s->rows >= (1 << 30) || s->features > 8192) return SSD_ERR_UNSUPPORTED;
  if (s->in_dtype == SSD_F32 && s->res_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  d->rows = (int)s->rows, d->F = (int)s->features, d->ng = (int)s->ngates;
  d->gs = d->ng && d->rows ? d->rows / d->ng : (d->rows ? d->rows : 1);
  d->eps = s->eps, d->scale = s->scale;
  return SSD_OK;
}

// Columns of a thread: 16 where rows divide into vectors, else 4, 8 above 2048
// columns and 16 above 4096 (512 threads at most).
int bn_cols(int F, bool vec) {
  return vec || F > 8 * kMaxThreads ? 16 : F > 4 * kMaxThreads ? 8 : 4;
}

// Blocks resident on an SM: 512 threads of them (100 to 128 registers each).
int bn_ctas(int nt) {
  const int n = 512 / nt;
  return n < 1 ? 1 : n > 16 ? 16 : n;
}

// Row ranges: as many blocks as are resident at once, each with the same number
// of consecutive rows; in the backward at least four while that still leaves
// two blocks an SM (each block adds a part to the gradients' sums: forward and
// backward of 600 x 1536 take 14.5 us, 16.5 with one row a block and 35 with 16).
void bn_grid(BnDims* d, bool vec, bool bwd) {
  const int sms = sm_count();
  d->nt = ceil_div(ceil_div(d->F, bn_cols(d->F, vec)), 32) * 32;
  d->R = ceil_div(d->rows, (int64_t)sms * bn_ctas(d->nt));
  if (bwd && d->R < 4) {
    const int few = ceil_div(d->rows, 2 * sms);
    d->R = few > 4 ? 4 : few > d->R ? few : d->R;
  }
  d->grid = ceil_div(d->rows, d->R);
}
// The backward's parts are counted for the scalar launch, which has the most
// blocks, so the size does not depend on addresses.
size_t bn_bwd_floats(BnDims d) {
  bn_grid(&d, false, true);
  const size_t a = ((size_t)2 * d.grid + (d.ng ? d.ng : 1)) * d.F;
  bn_grid(&d, true, true);
  const size_t b = ((size_t)2 * d.grid + (d.ng ? d.ng : 1)) * d.F;
  return a > b ? a : b;
}

struct BnPtrs {
  const void *r, *o;
  const float *w_pre, *w_post, *gate;
  const void *dh, *drout;
  void *rout, *h;  // forward outputs; the backward's dr and do
  float* part;
};

// Ring stages: what an SM's shared memory (200 KB of it) holds for its
// resident blocks, kMaxStages at most (one at the widest fp32 rows).
template <typename K>
cudaError_t bn_ring(K kern, BnDims* d, size_t stage, size_t* bytes) {
  *bytes = 0;
  d->S = 2;
  if (stage == 0) return cudaSuccess;
  const size_t fit = (size_t)200 * 1024 / bn_ctas(d->nt) / stage;
  d->S = fit < 1 ? 1 : fit > kMaxStages ? kMaxStages : (int)fit;
  *bytes = d->S * stage;
  // (a launch may have 48 KB without being allowed more, the blocks' sums included)
  return *bytes + sizeof(float2[2][16]) <= 48 * 1024
             ? cudaSuccess
             : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)*bytes);
}

template <typename Tio, typename Tres, int VEC, int EPT, bool FULL>
int bn_launch(BnDims d, const BnPtrs& p, bool bwd, cudaStream_t s) {
  const Tres* r = static_cast<const Tres*>(p.r);
  const Tio* o = static_cast<const Tio*>(p.o);
  size_t bytes;
  if (bwd) {
    auto kern = k_block_norm_bwd<Tio, Tres, VEC, EPT, FULL>;
    const size_t stage = (size_t)d.nt * Rows<Tio, Tres, VEC, EPT, FULL, 2, 2>::kSlot;
    if (bn_ring(kern, &d, stage, &bytes) != cudaSuccess) return SSD_ERR_CUDA;
    SSD_LAUNCH("k_block_norm_bwd", s,
               kern<<<d.grid, d.nt, bytes, s>>>(
                   r, o, p.w_pre, p.w_post, p.gate, static_cast<const Tio*>(p.dh),
                   static_cast<const Tres*>(p.drout), static_cast<Tres*>(p.rout),
                   static_cast<Tio*>(p.h), p.part, d));
  } else {
    auto kern = k_block_norm_fwd<Tio, Tres, VEC, EPT, FULL>;
    const size_t stage = (size_t)d.nt * Rows<Tio, Tres, VEC, EPT, FULL, 1, 1>::kSlot;
    if (bn_ring(kern, &d, stage, &bytes) != cudaSuccess) return SSD_ERR_CUDA;
    SSD_LAUNCH("k_block_norm_fwd", s,
               kern<<<d.grid, d.nt, bytes, s>>>(r, o, p.w_pre, p.w_post, p.gate,
                                                static_cast<Tres*>(p.rout),
                                                static_cast<Tio*>(p.h), d));
  }
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

template <typename Tio, typename Tres>
int bn_pick(const BnDims& d, const BnPtrs& p, int vec, bool bwd, cudaStream_t s) {
  if constexpr (sizeof(Tres) == 2) {
    if (vec == 8 && d.F == 16 * d.nt) return bn_launch<Tio, Tres, 8, 16, true>(d, p, bwd, s);
    if (vec == 8) return bn_launch<Tio, Tres, 8, 16, false>(d, p, bwd, s);
  }
  if (vec && d.F == 16 * d.nt) return bn_launch<Tio, Tres, 4, 16, true>(d, p, bwd, s);
  if (vec) return bn_launch<Tio, Tres, 4, 16, false>(d, p, bwd, s);
  if (bn_cols(d.F, vec) == 4) return bn_launch<Tio, Tres, 0, 4, false>(d, p, bwd, s);
  if (bn_cols(d.F, vec) == 8) return bn_launch<Tio, Tres, 0, 8, false>(d, p, bwd, s);
  return bn_launch<Tio, Tres, 0, 16, false>(d, p, bwd, s);
}

int bn_run(const BnDims& d, const ssd_block_norm_shape* sh, const BnPtrs& p, int vec, bool bwd,
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
  return bn_bwd_floats(d) * sizeof(float);
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
  const auto fits = [&](int w) {
    return d.F % w == 0 && vec_ok(o, d.F, ie, w) && vec_ok(h, d.F, ie, w) &&
           vec_ok(residual, d.F, re, w) && vec_ok(residual_out, d.F, re, w) &&
           vec_ok(w_pre, d.F, 4, 4) && vec_ok(w_post, d.F, 4, 4) && vec_ok(gate, d.F, 4, 4);
  };
  const int vec = re == 2 && fits(8) ? 8 : fits(4) ? 4 : 0;
  bn_grid(&d, vec, false);
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
  if (!workspace || off(workspace, 16) || workspace_bytes < bn_bwd_floats(d) * sizeof(float))
    return SSD_ERR_WORKSPACE;
  const auto fits = [&](int w) {
    return d.F % w == 0 && vec_ok(o, d.F, ie, w) && vec_ok(dh, d.F, ie, w) &&
           vec_ok(d_o, d.F, ie, w) && vec_ok(residual, d.F, re, w) &&
           vec_ok(dresidual_out, d.F, re, w) && vec_ok(dresidual, d.F, re, w) &&
           vec_ok(w_pre, d.F, 4, 4) && vec_ok(w_post, d.F, 4, 4) && vec_ok(gate, d.F, 4, 4);
  };
  const int vec = re == 2 && fits(8) ? 8 : fits(4) ? 4 : 0;
  bn_grid(&d, vec, true);
  const BnPtrs p{residual, o, w_pre, w_post, gate, dh, dresidual_out, dresidual, d_o,
                 static_cast<float*>(workspace)};
  const int e = bn_run(d, shape, p, vec, true, s);
  if (e != SSD_OK) return e;
  const dim3 grid(ceil_div(d.F, 32), 2 + d.ng < kMaxGridY ? 2 + d.ng : kMaxGridY);
  cudaError_t le;
  SSD_LAUNCH("k_block_norm_dw", s, le = launch_pdl(k_block_norm_dw, grid, 512, 0, s, p.part, w_post,
                                                   gate, dw_pre, dw_post, dgate, d));
  return le == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
