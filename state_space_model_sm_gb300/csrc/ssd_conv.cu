// Short causal depthwise convolution, the step in front of a layer's scan:
//     u[t, c] = bias[c] + sum_{k < K} w[c, k] x[t - K + 1 + k, c]
//     y = silu(u) or u,  silu(u) = u / (1 + e^-u)
// with x before position 0 taken from the carried state (the K - 1 inputs
// before the sequence, oldest first) or 0; its backward; and the single-token
// form, which shifts the state by one.
//
// All three are HBM streams: an element costs 2 K + ~8 operations against 4
// to 8 bytes, far below the machine's ratio.  Channels are contiguous, so a
// thread owns 4 consecutive channels (8 bytes of bf16, 16 of fp32; a warp's
// accesses are unbroken) and walks positions with the last K - 1 inputs in
// registers: every input is read once, plus K - 1 rows per segment.  The next
// rows are loaded while the current ones are used.
//
// Measured at 4 x 4096 x 1792, K = 4, silu, bf16: forward 25 us (4.7 TB/s, 0.69 of
// a plain copy's rate), backward 48 us (0.54) and 6 for the weights' sums; fp32:
// 0.77 over both.  bf16 is bound by issue as much as by memory (60 % and 52 % of
// the slots; 16 and 28 instructions an element, of which the taps are 2 and 6).
#include <cuda_bf16.h>

#include <type_traits>

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

// V channels as packed pairs, or as one value.
template <int V>
struct Lanes {
  using P = float2;
  static constexpr int N = V / 2;
};
template <>
struct Lanes<1> {
  using P = float;
  static constexpr int N = 1;
};
template <typename P>
__device__ __forceinline__ P splat(float v);
template <>
__device__ __forceinline__ float splat<float>(float v) { return v; }
template <>
__device__ __forceinline__ float2 splat<float2>(float v) { return f2(v); }

template <typename T, int V>
__device__ __forceinline__ void unpack_p(const Raw<T, V>& r, typename Lanes<V>::P (&p)[Lanes<V>::N]) {
  float f[V];
  unpack<T, V>(r, f);
#pragma unroll
  for (int i = 0; i < V; ++i) reinterpret_cast<float*>(p)[i] = f[i];
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack_p(const typename Lanes<V>::P (&p)[Lanes<V>::N]) {
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = reinterpret_cast<const float*>(p)[i];
  return pack<T, V>(f);
}

// The taps (and bias) of V channels.
template <int V, int K>
struct Taps {
  using P = typename Lanes<V>::P;
  static constexpr int N = Lanes<V>::N;
  P w[K][N], b[N];
  __device__ __forceinline__ Taps(const float* wp, const float* bias, int c0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t[4];
      const float* row = wp + (int64_t)(c0 + i) * K;
      if (K == 4 && V == 4) {
        *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(row);
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) t[k] = row[k];
      }
#pragma unroll
      for (int k = 0; k < K; ++k) reinterpret_cast<float*>(w[k])[i] = t[k];
      reinterpret_cast<float*>(b)[i] = bias ? bias[c0 + i] : 0.f;
    }
  }
  // sum over the taps of pair i of the window
  __device__ __forceinline__ P sum(const P (&win)[K][N], int i) const {
    P a = b[i];
#pragma unroll
    for (int k = 0; k < K; ++k) a = fma2(w[k][i], win[k][i], a);
    return a;
  }
};

// A thread's rows of one input from position t on, kU at a time.  Where its V
// channels are at least 4 bytes they are copied asynchronously into a ring in
// shared memory that only this thread reads (kStages - 1 groups ahead, no
// barrier and no registers); single bf16 channels go through registers, one
// group ahead (rows of 1791 bf16 channels take 1.5 times as long as 1792).
constexpr int kU = 4;
template <typename T, int V>
struct Feed {
  static constexpr bool kAsync = V * sizeof(T) >= 4;
  static constexpr int kStages = V * sizeof(T) > 8 ? 3 : 4;
  static constexpr int kBytes = kAsync ? kStages * kU * V * (int)sizeof(T) : 0;  // of a thread
  Raw<T, V>* ring;  // this thread's entry of position 0 of slot 0
  Raw<T, V> reg[kAsync ? 1 : kU], nxt[kAsync ? 1 : kU];
  const T* p;  // the next position to copy
  int64_t stride;
  int left, put, use;  // positions left to copy; slots

  __device__ __forceinline__ void fill() {
    if constexpr (kAsync) {
      Raw<T, V>* q = ring + put * kU * blockDim.x;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (u < left) cp_async<V * (int)sizeof(T)>(q + u * blockDim.x, p);
        p += stride;
      }
      cp_commit();
      put = put + 1 == kStages ? 0 : put + 1;
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (u < left) nxt[u] = ld_raw<T, V>(p);
        p += stride;
      }
    }
    left -= kU;
  }
  __device__ __forceinline__ void start(unsigned char* smem, const T* src, int64_t step, int count) {
    ring = reinterpret_cast<Raw<T, V>*>(smem) + threadIdx.x;
    p = src, stride = step, left = count, put = 0, use = kStages - 1;
  }
  static constexpr int kAhead = kAsync ? kStages - 1 : 1;  // groups copied ahead
  // Takes the next kU positions, copied by now (next_of), and starts a later copy.
  __device__ __forceinline__ void next() {
    if constexpr (kAsync) {
      use = use + 1 == kStages ? 0 : use + 1;
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) reg[u] = nxt[u];
    }
    fill();
  }
  __device__ __forceinline__ Raw<T, V> get(int u) const {
    if constexpr (kAsync) return ring[(use * kU + u) * blockDim.x];
    return reg[u];
  }
};

// The first copies, and then the next kU positions, of one or two feeds.  The feeds
// fill in turn from the first group on: copies complete in the order they were
// started, so leaving the last kStages - 2 of each in flight means that the group
// to be read has arrived in both (a thread reads only what it copied itself).
template <typename T, int V>
__device__ __forceinline__ void start_of(Feed<T, V>& a) {
#pragma unroll
  for (int i = 0; i < Feed<T, V>::kAhead; ++i) a.fill();
}
template <typename T, int V>
__device__ __forceinline__ void start_of(Feed<T, V>& a, Feed<T, V>& b) {
#pragma unroll
  for (int i = 0; i < Feed<T, V>::kAhead; ++i) {
    a.fill();
    b.fill();
  }
}
template <typename T, int V>
__device__ __forceinline__ void next_of(Feed<T, V>& a) {
  cp_wait<Feed<T, V>::kStages - 2>();
  a.next();
}
template <typename T, int V>
__device__ __forceinline__ void next_of(Feed<T, V>& a, Feed<T, V>& b) {
  cp_wait<2 * (Feed<T, V>::kStages - 2)>();
  a.next();
  b.next();
}

// Thread: V channels of one segment.  Work items are (batch, segment, vector)
// with the vector fastest, so a warp's accesses are contiguous.
template <typename Tin, typename Tout, int V, int K>
__global__ void __launch_bounds__(256)
    k_conv_fwd(const Tin* __restrict__ x, const float* __restrict__ w,
               const float* __restrict__ bias, const Tin* __restrict__ init,
               const int* __restrict__ lengths, Tout* __restrict__ y, Tin* __restrict__ final_state,
               ConvDims d) {
  using P = typename Lanes<V>::P;
  constexpr int N = Lanes<V>::N;
  const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t per_b = (int64_t)d.nseg * d.nvec;
  const int b = (int)(item / per_b);
  if (b >= d.B) return;
  const int rem = (int)(item - b * per_b), s = rem / d.nvec, c0 = (rem - s * d.nvec) * V;
  const int n = clamp_len(lengths, b, d.T);
  x += b * d.xb + c0;
  if (init) init += (int64_t)b * (K - 1) * d.C + c0;
  y += (int64_t)b * d.T * d.C + c0;

  const int t0 = s * d.seg, t1 = min(d.T, t0 + d.seg), tv = min(t1, n);
  extern __shared__ __align__(16) unsigned char smem[];
  Feed<Tin, V> in;
  if (t0 < tv) {
    in.start(smem, x + (int64_t)t0 * d.xs, d.xs, tv - t0);
    start_of(in);
  }
  if (s == 0 && final_state) {
    Tin* f = final_state + (int64_t)b * (K - 1) * d.C + c0;
    for (int j = 0; j < K - 1; ++j)
      st_raw<Tin, V>(f + (int64_t)j * d.C, ld_x<Tin, V, K>(x, init, d, n - (K - 1) + j));
  }
  if (t0 < tv) {
    const Taps<V, K> taps(w, bias, c0);
    P win[K][N];
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      unpack_p<Tin, V>(ld_x<Tin, V, K>(x, init, d, t0 - (K - 1) + k), win[k + 1]);
    Tout* o = y + (int64_t)t0 * d.C;
    for (int tb = t0; tb < tv; tb += kU) {
      next_of(in);
      auto step = [&](int u) {
        P out[N], xs[N];
        unpack_p<Tin, V>(in.get(u), xs);
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) win[k][i] = win[k + 1][i];
          win[K - 1][i] = xs[i];
          const P a = taps.sum(win, i);
          out[i] = d.silu ? mul2(a, sigmoid2(a)) : a;
        }
        st_raw<Tout, V>(o, pack_p<Tout, V>(out));
        o += d.C;
      };
      if (tb + kU <= tv) {
#pragma unroll
        for (int u = 0; u < kU; ++u) step(u);
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (tb + u < tv) step(u);
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
constexpr int kBwdWarps = 8, kBwdBlocksPerSm = 2;

template <typename Tin, typename Tout, int V, int K>
__global__ void __launch_bounds__(32 * kBwdWarps)
    k_conv_bwd(const Tin* __restrict__ x, const float* __restrict__ w,
               const float* __restrict__ bias, const Tin* __restrict__ init,
               const int* __restrict__ lengths, const Tin* __restrict__ dy,
               const Tin* __restrict__ dfinal, Tout* __restrict__ dx, Tout* __restrict__ dinit,
               float* __restrict__ part, ConvDims d, int nblk) {
  using P = typename Lanes<V>::P;
  constexpr int N = Lanes<V>::N;
  __shared__ float red[kBwdWarps][K + 1][32 * V];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v = blockIdx.y * 32 + lane, c0 = v * V;
  const int b = blockIdx.x / nblk, s = (blockIdx.x - b * nblk) * kBwdWarps + warp;
  P dw[K + 1][N];
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[k][i] = splat<P>(0.f);

  if (v < d.nvec && s < d.nseg) {
    const int n = clamp_len(lengths, b, d.T);
    x += b * d.xb + c0;
    dy += (int64_t)b * d.T * d.C + c0;
    dx += (int64_t)b * d.T * d.C + c0;
    const int64_t st0 = (int64_t)b * (K - 1) * d.C + c0;
    if (init) init += st0;
    const int t0 = s * d.seg, t1 = min(d.T, t0 + d.seg);
    const int te = t1 + K - 1;  // one past the last du this segment needs
    const int ti = min(te, n);  // .. and has
    extern __shared__ __align__(16) unsigned char smem[];
    Feed<Tin, V> fx, fg;
    fx.start(smem, x + (int64_t)t0 * d.xs, d.xs, ti - t0);
    fg.start(smem + Feed<Tin, V>::kBytes * blockDim.x, dy + (int64_t)t0 * d.C, d.C, ti - t0);
    start_of(fx, fg);
    const Taps<V, K> taps(w, bias, c0);
    P win[K][N], du[K][N];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) du[k][i] = splat<P>(0.f);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      unpack_p<Tin, V>(ld_x<Tin, V, K>(x, init, d, t0 - (K - 1) + k), win[k + 1]);
    for (int tb = t0; tb < te; tb += kU) {
      next_of(fx, fg);
      // EDGE: positions where du may be 0, dw not this segment's, or dx not of
      // this segment or also a state's
      auto step = [&](int u, auto edge) {
        constexpr bool EDGE = decltype(edge)::value;
        const int t = tb + u;
        const bool in = !EDGE || t < n;
        P xs[N], gs[N];
        unpack_p<Tin, V>(fx.get(u), xs);
        unpack_p<Tin, V>(fg.get(u), gs);
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) win[k][i] = win[k + 1][i], du[k][i] = du[k + 1][i];
          win[K - 1][i] = xs[i];
          P g = gs[i];
          if (d.silu) {
            const P a = taps.sum(win, i), sg = sigmoid2(a);
            g = mul2(g, fma2(mul2(sg, a), fma2(sg, splat<P>(-1.f), splat<P>(1.f)), sg));
          }
          du[K - 1][i] = in ? g : splat<P>(0.f);
          if (in && (!EDGE || t < t1)) {
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][i] = fma2(du[K - 1][i], win[k][i], dw[k][i]);
            dw[K][i] = add2(dw[K][i], du[K - 1][i]);
          }
        }
        const int sp = t - (K - 1);  // dx of this position is complete now
        if (EDGE && sp < t0 && s != 0) return;
        P o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          o[i] = splat<P>(0.f);
#pragma unroll
          for (int k = 0; k < K; ++k) o[i] = fma2(taps.w[k][i], du[K - 1 - k][i], o[i]);
        }
        if constexpr (EDGE) {
          const int j = t - n;  // x[sp] is entry j of the final state
          if (dfinal && j >= 0 && j < K - 1) {
            P f[N];
            unpack_p<Tin, V>(ld_raw<Tin, V>(dfinal + st0 + (int64_t)j * d.C), f);
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = add2(o[i], f[i]);
          }
          if (sp < 0) {
            if (dinit) st_raw<Tout, V>(dinit + st0 + (int64_t)t * d.C, pack_p<Tout, V>(o));
            return;
          }
        }
        st_raw<Tout, V>(dx + (int64_t)sp * d.C, pack_p<Tout, V>(o));
      };
      if (tb >= t0 + K - 1 && tb + kU <= min(t1, n)) {
#pragma unroll
        for (int u = 0; u < kU; ++u) step(u, std::false_type{});
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (tb + u < te) step(u, std::true_type{});
      }
    }
  }
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][k][lane * V + i] = reinterpret_cast<float*>(dw[k])[i];
  __syncthreads();
  // part (blocks, K + 1, C)
  const int nc = min(32 * V, d.C - (int)blockIdx.y * 32 * V);
  float* p = part + (int64_t)blockIdx.x * (K + 1) * d.C + (int64_t)blockIdx.y * 32 * V;
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
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
  float a = 0.f;
  if (c < C)
#pragma unroll 8
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
  const Taps<V, K> taps(w, bias, c0);
  typename Lanes<V>::P win[K][Lanes<V>::N], o[Lanes<V>::N];
#pragma unroll
  for (int k = 0; k < K; ++k) unpack_p<Tin, V>(raw[k], win[k]);
#pragma unroll
  for (int i = 0; i < Lanes<V>::N; ++i) {
    o[i] = taps.sum(win, i);
    if (d.silu) o[i] = mul2(o[i], sigmoid2(o[i]));
  }
#pragma unroll
  for (int k = 0; k < K - 1; ++k) st_raw<Tin, V>(st + (int64_t)k * d.C, raw[k + 1]);
  st_raw<Tout, V>(yo, pack_p<Tout, V>(o));
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
  if (s->batch >= 65536 || s->seqlen >= (1 << 30) || s->batch * s->seqlen >= ((int64_t)1 << 31) ||
      s->channels >= (1 << 20))
    return SSD_ERR_UNSUPPORTED;
  d->B = (int)s->batch, d->T = (int)s->seqlen, d->C = (int)s->channels;
  d->xs = s->x_row_stride ? s->x_row_stride : s->channels;
  d->xb = s->x_row_stride ? s->x_batch_stride : d->xs * d->T;
  d->silu = s->silu != 0;
  return SSD_OK;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Positions a thread walks, of 8 to 128, by the shortest modelled time: waves
// of resident threads, each as long as a segment and what it costs by itself
// (the K - 1 rows before it, the taps, one load's latency: about 12 positions).
// Against fixed segments of 16, 32 and 128, forward and backward: 70 us at
// 4 x 4096 x 1792 (92, 78, 84); forward at 1 x 512 x 1536: 6.3 us (8.3, 10.3, 22.6).
template <typename F>
void pick_segment(ConvDims* d, F&& waves) {
  int64_t best = -1;
  for (int seg = 8; seg <= 128; seg += 8) {
    const int nseg = ceil_div(d->T, seg);
    const int64_t cost = waves(nseg) * (seg + 12);
    if (best < 0 || cost < best) best = cost, d->seg = seg, d->nseg = nseg;
    if (nseg == 1) break;
  }
}
void fwd_segments(ConvDims* d) {  // four blocks of 256 threads an SM
  pick_segment(d, [&](int nseg) {
    const int64_t wave = 152 * 1024;
    return ((int64_t)d->B * nseg * d->nvec + wave - 1) / wave;
  });
}
void bwd_segments(ConvDims* d) {  // blocks of 32 vectors x 8 segments
  pick_segment(d, [&](int nseg) {
    const int64_t wave = 152 * kBwdBlocksPerSm;
    return ((int64_t)d->B * ceil_div(nseg, kBwdWarps) * ceil_div(d->nvec, 32) + wave - 1) / wave;
  });
}

// the backward's vector width and its blocks per sequence: shape-only, so
// the workspace query and the call agree
int bwd_parts(const ConvDims& d) { return d.B * ceil_div(d.nseg, kBwdWarps); }  // < 2^31: see conv_dims

template <typename Tin, typename Tout, int V>
int launch_fwd(ConvDims d, int K, const void* x, const float* w, const float* bias,
               const void* init, const int* lengths, void* y, void* final_state, cudaStream_t s) {
  d.nvec = d.C / V;
  fwd_segments(&d);
  const int64_t items = (int64_t)d.B * d.nseg * d.nvec, blocks = (items + 255) / 256;
  if (blocks > 0x7fffffff) return SSD_ERR_UNSUPPORTED;
  constexpr int smem = 256 * Feed<Tin, V>::kBytes;
  auto go = [&](auto kern) {
    if (smem > 48 * 1024) cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    SSD_LAUNCH("k_conv_fwd", s,
               kern<<<(unsigned)blocks, 256, smem, s>>>(
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
  const dim3 grid(nparts, ceil_div(d.nvec, 32));
  constexpr int smem = 2 * 32 * kBwdWarps * Feed<Tin, V>::kBytes;
  auto go = [&](auto kern) {
    if (smem + 20 * 1024 > 48 * 1024)  // with the sums, 20 KB at most
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    SSD_LAUNCH("k_conv_bwd", s,
               kern<<<grid, 32 * kBwdWarps, smem, s>>>(
                   static_cast<const Tin*>(x), w, bias, static_cast<const Tin*>(init), lengths,
                   static_cast<const Tin*>(dy), static_cast<const Tin*>(dfinal),
                   static_cast<Tout*>(dx), static_cast<Tout*>(dinit), part, d, nblk));
  };
  if (K == 2) go(k_conv_bwd<Tin, Tout, V, 2>);
  if (K == 3) go(k_conv_bwd<Tin, Tout, V, 3>);
  if (K == 4) go(k_conv_bwd<Tin, Tout, V, 4>);
  const dim3 rg(ceil_div(d.C, 32), K + 1);
  if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;
  cudaError_t e;
  SSD_LAUNCH("k_conv_dw", s,
             e = launch_pdl(k_conv_dw, rg, 256, 0, s, part, dw, dbias, nparts, d.C, K));
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
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
  if (init_state && final_state) {  // the final state is written before the initial one is used up
    const uintptr_t a = reinterpret_cast<uintptr_t>(init_state);
    const uintptr_t b = reinterpret_cast<uintptr_t>(final_state);
    if ((a > b ? a - b : b - a) < (uintptr_t)d.B * (K - 1) * d.C * ie) return SSD_ERR_INVALID_ARG;
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = d.C % 4 == 0 && vec_ok(x, d.xs, ie, 4) && vec_ok(x, d.xb, ie, 4) &&
                   vec_ok(init_state, d.C, ie, 4) && vec_ok(final_state, d.C, ie, 4) &&
                   vec_ok(y, d.C, oe, 4) && vec_ok(w, 4, 4, 4);
#define SSD_GO(TI, TO, V) \
  launch_fwd<TI, TO, V>(d, K, x, w, bias, init_state, lengths, y, final_state, s)
  if (ie == 4) return vec ? SSD_GO(float, float, 4) : SSD_GO(float, float, 1);
  if (oe == 4) return vec ? SSD_GO(bf16, float, 4) : SSD_GO(bf16, float, 1);
  return vec ? SSD_GO(bf16, bf16, 4) : SSD_GO(bf16, bf16, 1);
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
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  const bool vec = d.C % 4 == 0 && vec_ok(x, d.xs, ie, 4) && vec_ok(x, d.xb, ie, 4) && vec_ok(init_state, d.C, ie, 4) &&
                   vec_ok(dy, d.C, ie, 4) && vec_ok(dfinal_state, d.C, ie, 4) &&
                   vec_ok(dx, d.C, oe, 4) && vec_ok(dinit_state, d.C, oe, 4) && vec_ok(w, 4, 4, 4);
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
  const bool vec = d.C % 4 == 0 && vec_ok(x, d.xs, ie, 4) && vec_ok(state, d.C, ie, 4) &&
                   vec_ok(y, d.C, oe, 4) && vec_ok(w, 4, 4, 4);
#define SSD_GO(TI, TO, V) \
  launch_step<TI, TO, V>(d, K, x, state, w, bias, slots, nslots, y, s)
  if (ie == 4) return vec ? SSD_GO(float, float, 4) : SSD_GO(float, float, 1);
  if (oe == 4) return vec ? SSD_GO(bf16, float, 4) : SSD_GO(bf16, float, 1);
  return vec ? SSD_GO(bf16, bf16, 4) : SSD_GO(bf16, bf16, 1);
#undef SSD_GO
}

}  // extern "C"
