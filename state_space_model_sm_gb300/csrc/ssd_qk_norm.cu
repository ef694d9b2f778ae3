// Norm of queries and keys per head, with the rotation of positions in the same pass
// (layer operator in front of the scans: the keys and queries of the delta rule, the B
// and C of the SSD scan).  For a head's row x of D values
//     n = x rstd w,   rstd = 1 / sqrt(mean x^2 + eps)   (l2: sum)
// and pairs (a, b) of n's first R columns turned by f = position * freq:
//     a' = a cos f - b sin f,   b' = b cos f + a sin f.
// Backward: g is the gradient turned by -f;  dw += g x rstd,
//     dx = rstd (g w - xhat mean(g w xhat))             (l2: sum).
//
// Bandwidth-bound: a row is read and written once (backward: two reads, one write).  A
// head's row lies on LPH lanes, NS pieces of V columns of each half of its pairs a
// lane, so that both members of a pair are in one lane; a warp takes the heads of one
// token, 32 / LPH at a time, and forms the token's sines and cosines once for them all.
// 4 x 4096 tokens of 36 heads of 128, bf16: forward 61 us, 4.9 TB/s of the rows; backward
// 99 us, 4.6 TB/s; 2 x 8192 tokens of 32 heads without weights and rotation 52 us, 5.2 TB/s.
//
// Angles: position * freq loses the fraction of a turn in fp32 from some thousand
// radians on.  Here freq / 2 pi is a 64-bit fraction of a turn, formed once a block from
// the bits of freq and of 1 / 2 pi, and the angle is the 64-bit integer product with
// the position, whose overflow is whole turns: exact to 2^-31 turns for every int32, and
// then rounded to a float's 24 bits, 2^-26 turns at most.
#include <cuda_bf16.h>

#include "layer_math.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace {

using namespace lm;
using bf16 = __nv_bfloat16;

struct QkDims {
  int B, T, HQ, HK, D, R;
  int parts;      // parts that a token's heads are split into, a warp each
  int64_t units;  // tokens * parts
  int64_t qs, qb, ks, kb;
  float eps, inv;  // inv: 1 / D, or 1 with l2
  int interleaved;
};

constexpr int kQkThreads = 128;
constexpr int kQkWarps = kQkThreads / 32;

// f / 2 pi in turns, modulo 1, times 2^64: m 2^e / 2 pi with a 24-bit m, by the first
// 128 bits of 1 / 2 pi.  They reach as far as |f| < 2^20; a larger, infinite or NaN
// frequency is kNoTurn, whose angles are NaN.
constexpr uint64_t kNoTurn = 0x8000000000000001u;
__device__ __forceinline__ uint64_t turns(float f) {
  const uint32_t w = __float_as_uint(f);
  const int ex = (int)((w >> 23) & 0xffu);
  if (ex >= 147) return kNoTurn;
  const uint32_t m = ex ? (w & 0x7fffffu) | 0x800000u : w & 0x7fffffu;
  const int e = (ex ? ex : 1) - 150;
  // m / 2 pi * 2^128 in five words
  constexpr uint32_t c[4] = {0x7d4d3770u, 0x7f09d5f4u, 0x9391054au, 0x28be60dbu};
  uint32_t p[5];
  uint64_t carry = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    carry += (uint64_t)m * c[i];
    p[i] = (uint32_t)carry;
    carry >>= 32;
  }
  p[4] = (uint32_t)carry;
  // bits [s, s + 64), s = 64 - e
  const int s = 64 - e;
  uint64_t r = 0;
  if (s < 160) {
    const int q = s >> 5, o = s & 31;
    uint32_t x[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      x[i] = 0;
#pragma unroll
      for (int j = 0; j < 5; ++j)
        if (j == q + i) x[i] = p[j];
    }
    const uint32_t lo = __funnelshift_r(x[0], x[1], o), hi = __funnelshift_r(x[1], x[2], o);
    r = (uint64_t)hi << 32 | lo;
  }
  r = w >> 31 ? 0 - r : r;
  return r == kNoTurn ? r + 1 : r;  // (2^-64 of a turn off)
}

__device__ __forceinline__ void rotation(uint64_t turn, int pos, float* sn, float* cs) {
  const uint64_t t = turn * (uint64_t)(int64_t)pos;
  if (turn == kNoTurn) {
    *sn = *cs = __int_as_float(0x7fffffff);
    return;
  }
  sincospif((float)(int32_t)(uint32_t)(t >> 32) * 4.656612873077393e-10f, sn, cs);  // 2^-31
}

// The two columns of piece s (first of V) of a head, and whether it is turned; b < 0:
// there is no second one.
template <int V>
__device__ __forceinline__ void columns(const QkDims& d, int s, int* a, int* b, bool* on) {
  const int hr = d.R >> 1, c = s * V;
  if (V > 1 && d.interleaved) {  // pairs lie inside a piece
    *a = c, *b = c + (d.D >> 1);
    *on = true;
    return;
  }
  *on = c < hr;
  if (c < hr) {
    *a = d.interleaved ? 2 * c : c;
    *b = d.interleaved ? 2 * c + 1 : c + hr;
  } else {
    const int rest = (d.D - d.R + 1) >> 1;
    *a = d.R + c - hr;
    *b = *a + rest;
    if (*b >= d.D) *b = -1;
  }
}

// Where a lane's pieces lie: first columns (a < 0: no piece), whether they are turned, and
// the first of their pairs (interleaved pieces of two pairs a column: of a's; b's first is
// D / 4 further).
template <int V, int NS>
struct Lane {
  int a[NS], b[NS], pair[NS];
  bool on[NS];
};

template <int V, int NS>
__device__ __forceinline__ void set_lane(const QkDims& d, int sl, int lph, Lane<V, NS>* L) {
  const int pieces = V > 1 ? d.D / (2 * V) : (d.R >> 1) + ((d.D - d.R + 1) >> 1);
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    const int s = n * lph + sl;
    L->a[n] = L->b[n] = -1;
    L->on[n] = false;
    if (s < pieces) columns<V>(d, s, &L->a[n], &L->b[n], &L->on[n]);
    if (d.R == 0) L->on[n] = false;
    L->pair[n] = V > 1 && d.interleaved ? s * V / 2 : s * V;
  }
}

// Shared memory: what a frequency turns a step by, the weights (1 where there are none),
// and for each warp its token's sines and cosines.  Pairs that do not turn (columns from
// R on of interleaved pieces) have sine 0 and cosine 1.
struct QkSmem {
  uint64_t* turn;
  float *w, *rot;
  int pairs;  // a multiple of 4
};
__host__ __device__ inline int qk_pairs(int D) { return (D / 2 + 3) / 4 * 4; }
__host__ __device__ inline size_t qk_smem(int D, int R) {
  return (R ? (size_t)qk_pairs(D) * (8 + kQkWarps * 8) : 0) + (size_t)2 * ((D + 3) / 4 * 4) * 4;
}
__device__ __forceinline__ QkSmem qk_tables(const QkDims& d, unsigned char* smem, const float* freq,
                                            const float* w_q, const float* w_k) {
  QkSmem m;
  m.pairs = qk_pairs(d.D);
  m.w = reinterpret_cast<float*>(smem);
  const int dw = (d.D + 3) / 4 * 4;
  m.turn = reinterpret_cast<uint64_t*>(m.w + 2 * dw);
  m.rot = reinterpret_cast<float*>(m.turn + m.pairs) + (threadIdx.x >> 5) * 2 * m.pairs;
  for (int i = threadIdx.x; i < d.D; i += kQkThreads) {
    m.w[i] = w_q ? w_q[i] : 1.f;
    m.w[dw + i] = w_k ? w_k[i] : 1.f;
  }
  if (d.R)
    for (int i = threadIdx.x; i < m.pairs; i += kQkThreads)
      m.turn[i] = 2 * i < d.R ? turns(freq[i]) : 0;
  return m;
}
// V values from p on, in pieces of up to 4 (p is then 16-byte aligned).
template <int V>
__device__ __forceinline__ void from_table(const float* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = p[0];
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + j);
      f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_piece(T* p, int c, const float (&f)[V]) {
  if (c >= 0) st_raw<T, V>(p + c, pack<T, V>(f));
}
// (a, b) turned: by the angle (DIR 1) or back (DIR -1).
template <int DIR, int V>
__device__ __forceinline__ void turn(bool inter, const float (&sn)[V], const float (&cs)[V],
                                     float (&a)[V], float (&b)[V]) {
  if (V > 1 && inter) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float s0 = DIR * sn[j], s1 = DIR * sn[V / 2 + j];
      const float x = a[2 * j], y = a[2 * j + 1], z = b[2 * j], w = b[2 * j + 1];
      a[2 * j] = fmaf(x, cs[j], -y * s0), a[2 * j + 1] = fmaf(y, cs[j], x * s0);
      b[2 * j] = fmaf(z, cs[V / 2 + j], -w * s1), b[2 * j + 1] = fmaf(w, cs[V / 2 + j], z * s1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float s = DIR * sn[j], x = a[j], y = b[j];
      a[j] = fmaf(x, cs[j], -y * s), b[j] = fmaf(y, cs[j], x * s);
    }
  }
}

// A unit's token and position, its rows of q and k, and the heads (queries, then keys) of
// its part.
struct Unit {
  int row, pos, h0, h1;
  int64_t q, k;  // elements from the inputs' start to the token's first head
};
__device__ __forceinline__ Unit unit(const QkDims& d, int u, const int* positions) {
  Unit x;
  x.row = d.parts == 1 ? u : u / d.parts;
  const int part = u - x.row * d.parts, n = d.HQ + d.HK;
  x.h0 = d.parts == 1 ? 0 : (int)((int64_t)n * part / d.parts);
  x.h1 = d.parts == 1 ? n : (int)((int64_t)n * (part + 1) / d.parts);
  const int b = x.row / d.T, t = x.row - b * d.T;
  x.q = b * d.qb + t * d.qs;
  x.k = b * d.kb + t * d.ks;
  x.pos = d.R == 0 ? 0 : positions ? positions[x.row] : t;
  return x;
}

// The raw pieces of a head's row.
template <typename T, int V, int NS>
struct Row {
  Raw<T, V> a[NS], b[NS];
  __device__ __forceinline__ void load(const T* p, const Lane<V, NS>& L) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      a[n] = L.a[n] >= 0 ? ld_raw<T, V>(p + L.a[n]) : zero_raw<T, V>();
      b[n] = L.b[n] >= 0 ? ld_raw<T, V>(p + L.b[n]) : zero_raw<T, V>();
    }
  }
};

// The weights of queries (kind 0) or keys in a lane's columns.
template <int V, int NS>
__device__ __forceinline__ void weights(const QkDims& d, const QkSmem& m, const Lane<V, NS>& L, int kind,
                                        float (&wa)[NS][V], float (&wb)[NS][V]) {
  const float* w = m.w + kind * ((d.D + 3) / 4 * 4);
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    from_table<V>(w + max(L.a[n], 0), wa[n]);
    from_table<V>(w + max(L.b[n], 0), wb[n]);
  }
}

// The sines and cosines of a token in a lane's columns: each formed by one lane of the
// warp, handed on through shared memory.
template <int V, int NS>
__device__ __forceinline__ void rotations(const QkDims& d, const QkSmem& m, const Lane<V, NS>& L, int pos,
                                          float (&sn)[NS][V], float (&cs)[NS][V]) {
  if (d.R == 0) return;
  __syncwarp();  // the last token's are read
  for (int i = threadIdx.x & 31; i < m.pairs; i += 32) {
    float a = 0.f, b = 1.f;
    if (2 * i < d.R) rotation(m.turn[i], pos, &a, &b);
    m.rot[i] = a;
    m.rot[m.pairs + i] = b;
  }
  __syncwarp();
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (L.on[n]) {
      if constexpr (V > 1) {
        if (d.interleaved) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const int i = L.pair[n] + j, k = i + (d.D >> 2);
            sn[n][j] = m.rot[i], cs[n][j] = m.rot[m.pairs + i];
            sn[n][V / 2 + j] = m.rot[k], cs[n][V / 2 + j] = m.rot[m.pairs + k];
          }
          continue;
        }
      }
      from_table<V>(m.rot + L.pair[n], sn[n]);
      from_table<V>(m.rot + m.pairs + L.pair[n], cs[n]);
    }
}

template <typename T, typename TO, int V, int LPH, int NS>
__global__ void __launch_bounds__(kQkThreads, NS == 1 ? 6 : 1)
    k_qk_norm_fwd(QkDims d, const T* __restrict__ q, const T* __restrict__ k,
                  const float* __restrict__ w_q, const float* __restrict__ w_k,
                  const float* __restrict__ freq, const int* __restrict__ positions,
                  TO* __restrict__ q_out, TO* __restrict__ k_out) {
  constexpr int HP = 32 / LPH;  // heads of a warp at a time
  const int lane = threadIdx.x & 31, seg = lane / LPH, sl = lane % LPH;
  const int step = gridDim.x * kQkWarps;
  const bool inter = d.interleaved != 0;
  extern __shared__ __align__(16) unsigned char tables[];
  Lane<V, NS> L;
  set_lane<V, NS>(d, sl, LPH, &L);
  const QkSmem m = qk_tables(d, tables, freq, w_q, w_k);
  __syncthreads();
  for (int64_t u = (int64_t)blockIdx.x * kQkWarps + (threadIdx.x >> 5); u < d.units; u += step) {
    const Unit x = unit(d, (int)u, positions);
    float sn[NS][V], cs[NS][V];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {  // queries, keys
      const int base = kind ? d.HQ : 0;
      const int lo = max(x.h0, base) - base, hi = (kind ? x.h1 : min(x.h1, d.HQ)) - base;
      if (lo >= hi) continue;
      const T* in = (kind ? k + x.k : q + x.q);
      TO* out = kind ? k_out + (int64_t)x.row * d.HK * d.D : q_out + (int64_t)x.row * d.HQ * d.D;
      Row<T, V, NS> next;
      next.load(in + (int64_t)min(lo + seg, hi - 1) * d.D, L);
      float wa[NS][V], wb[NS][V];
      weights<V, NS>(d, m, L, kind, wa, wb);
      if (kind == 0 || x.h0 >= d.HQ) rotations<V, NS>(d, m, L, x.pos, sn, cs);
      for (int h = lo + seg; h - seg < hi; h += HP) {
        const Row<T, V, NS> now = next;  // the next head's row is on its way
        if (h + HP - seg < hi) next.load(in + (int64_t)min(h + HP, hi - 1) * d.D, L);
        float a[NS][V], b[NS][V], ss = 0.f;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          unpack<T, V>(now.a[n], a[n]);
          unpack<T, V>(now.b[n], b[n]);
#pragma unroll
          for (int j = 0; j < V; ++j) ss = fmaf(a[n][j], a[n][j], fmaf(b[n][j], b[n][j], ss));
        }
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rs = rsqrtf(fmaf(ss, d.inv, d.eps));
        TO* to = out + (int64_t)h * d.D;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            a[n][j] *= rs * wa[n][j];
            b[n][j] *= rs * wb[n][j];
          }
          if (L.on[n]) turn<1, V>(inter, sn[n], cs[n], a[n], b[n]);
          if (h < hi) {
            store_piece<TO, V>(to, L.a[n], a[n]);
            store_piece<TO, V>(to, L.b[n], b[n]);
          }
        }
      }
    }
  }
}

// part (gridDim.x, 2, D): each block's sums of dw_q and dw_k.
template <typename T, typename TO, int V, int LPH, int NS>
__global__ void __launch_bounds__(kQkThreads, NS == 1 ? 4 : 1)
    k_qk_norm_bwd(QkDims d, const T* __restrict__ q, const T* __restrict__ k,
                  const float* __restrict__ w_q, const float* __restrict__ w_k,
                  const float* __restrict__ freq, const int* __restrict__ positions,
                  const T* __restrict__ dqo, const T* __restrict__ dko, TO* __restrict__ dq,
                  TO* __restrict__ dk, float* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char tables[];
  float* const sums = reinterpret_cast<float*>(tables + qk_smem(d.D, d.R));  // (warps, 2, D)
  const int lane = threadIdx.x & 31, seg = lane / LPH, sl = lane % LPH, warp = threadIdx.x >> 5;
  constexpr int HP = 32 / LPH;
  const int step = gridDim.x * kQkWarps;
  const bool inter = d.interleaved != 0;
  Lane<V, NS> L;
  set_lane<V, NS>(d, sl, LPH, &L);
  const QkSmem tb = qk_tables(d, tables, freq, w_q, w_k);
  __syncthreads();
  float ga[2][NS][V], gb[2][NS][V];  // sums of dw
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int j = 0; j < V; ++j) ga[kind][n][j] = gb[kind][n][j] = 0.f;
  for (int64_t u = (int64_t)blockIdx.x * kQkWarps + warp; u < d.units; u += step) {
    const Unit x = unit(d, (int)u, positions);
    float sn[NS][V], cs[NS][V];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int base = kind ? d.HQ : 0;
      const int lo = max(x.h0, base) - base, hi = (kind ? x.h1 : min(x.h1, d.HQ)) - base;
      if (lo >= hi) continue;
      const T* in = (kind ? k + x.k : q + x.q);
      const int64_t dense = (int64_t)x.row * (kind ? d.HK : d.HQ) * d.D;
      const T* up = (kind ? dko : dqo) + dense;
      TO* out = (kind ? dk : dq) + dense;
      Row<T, V, NS> nx, ng;
      nx.load(in + (int64_t)min(lo + seg, hi - 1) * d.D, L);
      ng.load(up + (int64_t)min(lo + seg, hi - 1) * d.D, L);
      float wa[NS][V], wb[NS][V];
      weights<V, NS>(d, tb, L, kind, wa, wb);
      if (kind == 0 || x.h0 >= d.HQ) rotations<V, NS>(d, tb, L, x.pos, sn, cs);
      for (int h = lo + seg; h - seg < hi; h += HP) {
        const Row<T, V, NS> cx = nx, cg = ng;  // the next head's rows are on their way
        if (h + HP - seg < hi) {
          nx.load(in + (int64_t)min(h + HP, hi - 1) * d.D, L);
          ng.load(up + (int64_t)min(h + HP, hi - 1) * d.D, L);
        }
        float a[NS][V], b[NS][V], g[NS][V], f[NS][V], ss = 0.f, dot = 0.f;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          unpack<T, V>(cx.a[n], a[n]);
          unpack<T, V>(cx.b[n], b[n]);
          unpack<T, V>(cg.a[n], g[n]);
          unpack<T, V>(cg.b[n], f[n]);
          if (L.on[n]) turn<-1, V>(inter, sn[n], cs[n], g[n], f[n]);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            ss = fmaf(a[n][j], a[n][j], fmaf(b[n][j], b[n][j], ss));
            dot = fmaf(a[n][j] * wa[n][j], g[n][j], fmaf(b[n][j] * wb[n][j], f[n][j], dot));
          }
        }
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float rs = rsqrtf(fmaf(ss, d.inv, d.eps));
        const float m = dot * rs * d.inv * rs;  // rstd mean(g w xhat)
        const float keep = h < hi ? rs : 0.f;
        TO* to = out + (int64_t)h * d.D;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            ga[kind][n][j] = fmaf(g[n][j], a[n][j] * keep, ga[kind][n][j]);
            gb[kind][n][j] = fmaf(f[n][j], b[n][j] * keep, gb[kind][n][j]);
            a[n][j] = rs * fmaf(-a[n][j], m, g[n][j] * wa[n][j]);
            b[n][j] = rs * fmaf(-b[n][j], m, f[n][j] * wb[n][j]);
          }
          if (h < hi) {
            store_piece<TO, V>(to, L.a[n], a[n]);
            store_piece<TO, V>(to, L.b[n], b[n]);
          }
        }
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float a = ga[kind][n][j], b = gb[kind][n][j];
#pragma unroll
        for (int o = LPH; o < 32; o <<= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (seg == 0) {
          float* s = sums + (warp * 2 + kind) * d.D;
          if (L.a[n] >= 0) s[L.a[n] + j] = a;
          if (L.b[n] >= 0) s[L.b[n] + j] = b;
        }
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * d.D; i += kQkThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kQkWarps; ++w) s += sums[w * 2 * d.D + i];
    part[(int64_t)blockIdx.x * 2 * d.D + i] = s;
  }
}

// dw_q and dw_k: 32 columns a block, 32 ranges of the blocks' sums, in a fixed order.
__global__ void __launch_bounds__(1024)
    k_qk_norm_dw(const float* __restrict__ part, int blocks, int D, float* __restrict__ dw_q,
                 float* __restrict__ dw_k) {
  __shared__ float s[32][32];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
  float a = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int i = r; i < blocks; i += 32) a += part[(int64_t)i * 2 * D + c];
  }
  s[r][lane] = a;
  __syncthreads();
  if (r == 0 && c < 2 * D) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += s[i][lane];
    float* to = c < D ? dw_q : dw_k;
    if (to) to[c < D ? c : c - D] = a;
  }
}

// ---------------------------------------------------------------------- host

bool off(const void* p, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(esize - 1)) != 0;
}

// Blocks an SM of the forward (at most; 8 and 16: 8 % and 0 % slower) and of the backward,
// whose sums each block holds (2 and 8: forward and backward together 25 % and 3 % slower).
constexpr int kFwdBlocksPerSm = 12, kBwdBlocksPerSm = 4;

int qk_dims(const ssd_qk_norm_shape* s, QkDims* d) {
  if (!s || s->batch < 1 || s->seqlen < 1 || s->q_heads < 1 || s->k_heads < 1 || s->headdim < 1 ||
      s->rotary < 0 || s->rotary % 2 != 0 || s->rotary > s->headdim || !(s->eps > 0.f))
    return SSD_ERR_INVALID_ARG;
  if ((s->in_dtype != SSD_F32 && s->in_dtype != SSD_BF16) ||
      (s->out_dtype != SSD_F32 && s->out_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  if (s->in_dtype == SSD_F32 && s->out_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->headdim > 1024 || s->q_heads >= 65536 || s->k_heads >= 65536 || s->batch >= (1 << 30) ||
      s->seqlen >= (1 << 30) ||
      s->batch * s->seqlen >= 0x7fffffffLL / (s->q_heads + s->k_heads))
    return SSD_ERR_UNSUPPORTED;
  const int64_t qw = s->q_heads * s->headdim, kw = s->k_heads * s->headdim;
  if ((s->q_row_stride && s->q_row_stride < qw) || (s->k_row_stride && s->k_row_stride < kw) ||
      s->q_batch_stride < 0 || s->k_batch_stride < 0)
    return SSD_ERR_INVALID_ARG;
  d->B = (int)s->batch, d->T = (int)s->seqlen, d->HQ = (int)s->q_heads, d->HK = (int)s->k_heads;
  d->D = (int)s->headdim, d->R = (int)s->rotary;
  d->qs = s->q_row_stride ? s->q_row_stride : qw;
  d->ks = s->k_row_stride ? s->k_row_stride : kw;
  d->qb = s->q_row_stride ? s->q_batch_stride : d->qs * d->T;
  d->kb = s->k_row_stride ? s->k_batch_stride : d->ks * d->T;
  d->eps = s->eps, d->inv = s->l2 ? 1.f : 1.f / (float)s->headdim;
  d->interleaved = s->interleaved;
  return SSD_OK;
}

// A token's heads are split where there are fewer tokens than 16 warps an SM, down to
// the `per` heads that a warp takes at a time (64 tokens of 40 heads of 128: 6.1 us, 8.4
// whole; 1024 tokens of 32: 6.2 and 8.2).
void split(QkDims* d, int per) {
  const int64_t rows = (int64_t)d->B * d->T, n = d->HQ + d->HK;
  int64_t parts = kRuleSms * 16 / rows;
  const int64_t most = (n + per - 1) / per;
  parts = parts < 1 ? 1 : parts > most ? most : parts;
  d->parts = (int)parts;
  d->units = rows * parts;
}

// Blocks of the backward for any way of splitting: its workspace.
int64_t bwd_blocks(const QkDims& d) {
  const int64_t most = (int64_t)sm_count() * kBwdBlocksPerSm;
  const int64_t b = ((int64_t)d.B * d.T * (d.HQ + d.HK) + kQkWarps - 1) / kQkWarps;
  return b < most ? b : most;
}

struct QkPtrs {
  const void *q, *k;
  const float *w_q, *w_k, *freq;
  const int32_t* positions;
  void *q_out, *k_out;            // forward
  const void *dqo, *dko;          // backward
  void *dq, *dk;
  float *dw_q, *dw_k, *part;
};

template <typename T, typename TO, int V, int LPH, int NS>
int qk_launch(QkDims d, const QkPtrs& p, bool bwd, cudaStream_t s) {
  split(&d, 32 / LPH);
  const T *q = static_cast<const T*>(p.q), *k = static_cast<const T*>(p.k);
  int64_t blocks = (d.units + kQkWarps - 1) / kQkWarps;
  if (!bwd) {
    const int64_t most = (int64_t)sm_count() * kFwdBlocksPerSm;
    blocks = blocks < most ? blocks : most;
    SSD_LAUNCH("k_qk_norm_fwd", s,
               k_qk_norm_fwd<T, TO, V, LPH, NS><<<(unsigned)blocks, kQkThreads, qk_smem(d.D, d.R), s>>>(
                   d, q, k, p.w_q, p.w_k, p.freq, p.positions, static_cast<TO*>(p.q_out),
                   static_cast<TO*>(p.k_out)));
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
  }
  const int64_t most = bwd_blocks(d);
  blocks = blocks < most ? blocks : most;
  float* part = p.w_q || p.w_k ? p.part : nullptr;
  const size_t smem = qk_smem(d.D, d.R) + (part ? kQkWarps * 2 * d.D * sizeof(float) : 0);
  // the limit of the largest head, so that calls at the same time set the same
  constexpr int kMaxD = 1024;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k_qk_norm_bwd<T, TO, V, LPH, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(qk_smem(kMaxD, kMaxD) + kQkWarps * 2 * kMaxD * sizeof(float))) != cudaSuccess)
    return SSD_ERR_CUDA;
  SSD_LAUNCH("k_qk_norm_bwd", s,
             k_qk_norm_bwd<T, TO, V, LPH, NS>
             <<<(unsigned)blocks, kQkThreads, smem, s>>>(
                 d, q, k, p.w_q, p.w_k, p.freq, p.positions, static_cast<const T*>(p.dqo),
                 static_cast<const T*>(p.dko), static_cast<TO*>(p.dq), static_cast<TO*>(p.dk), part));
  if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;
  if (!part) return SSD_OK;
  SSD_LAUNCH("k_qk_norm_dw", s,
             k_qk_norm_dw<<<(unsigned)((2 * d.D + 31) / 32), 1024, 0, s>>>(part, (int)blocks, d.D,
                                                                          p.dw_q, p.dw_k));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// Pieces of 16 bytes where every row and both halves of the pairs are made of them,
// else single columns; the fewest lanes that hold a row.
template <typename T, typename TO>
int qk_pick(const QkDims& d, const QkPtrs& p, bool wide, bool bwd, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (wide) {
    const int n = d.D / (2 * V);
    if (n <= 4) return qk_launch<T, TO, V, 4, 1>(d, p, bwd, s);
    if (n <= 8) return qk_launch<T, TO, V, 8, 1>(d, p, bwd, s);
    if (n <= 16) return qk_launch<T, TO, V, 16, 1>(d, p, bwd, s);
    if (n <= 32) return qk_launch<T, TO, V, 32, 1>(d, p, bwd, s);
    if (n <= 64) return qk_launch<T, TO, V, 32, 2>(d, p, bwd, s);
    if constexpr (V == 4) return qk_launch<T, TO, V, 32, 4>(d, p, bwd, s);
  }
  const int n = (d.R >> 1) + ((d.D - d.R + 1) >> 1);
  if (n <= 16) return qk_launch<T, TO, 1, 16, 1>(d, p, bwd, s);
  if (n <= 64) return qk_launch<T, TO, 1, 32, 2>(d, p, bwd, s);
  return qk_launch<T, TO, 1, 32, 16>(d, p, bwd, s);
}

int qk_run(const ssd_qk_norm_shape* shape, const QkDims& d, const QkPtrs& p, bool bwd, void* stream) {
  const int ie = shape->in_dtype == SSD_BF16 ? 2 : 4;
  const bool ob = shape->out_dtype == SSD_BF16;
  const int V = 16 / ie;
  bool wide = d.D % (2 * V) == 0 && (d.interleaved || d.R % (2 * V) == 0) && d.qs % V == 0 &&
              d.qb % V == 0 && d.ks % V == 0 && d.kb % V == 0;
  const void* ins[4] = {p.q, p.k, p.dqo, p.dko};
  const void* outs[4] = {p.q_out, p.k_out, p.dq, p.dk};
  for (int i = 0; i < 4; ++i) wide = wide && !off(ins[i], 16) && !off(outs[i], 16);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (ie == 4) return qk_pick<float, float>(d, p, wide, bwd, s);
  return ob ? qk_pick<bf16, bf16>(d, p, wide, bwd, s) : qk_pick<bf16, float>(d, p, wide, bwd, s);
}

int qk_check(const ssd_qk_norm_shape* shape, QkDims* d, const QkPtrs& p) {
  const int st = qk_dims(shape, d);
  if (st != SSD_OK) return st;
  const int e = shape->in_dtype == SSD_BF16 ? 2 : 4;
  if (!p.q || !p.k || (d->R > 0 && !p.freq)) return SSD_ERR_INVALID_ARG;
  if (off(p.q, e) || off(p.k, e) || off(p.w_q, 4) || off(p.w_k, 4) || off(p.freq, 4) ||
      off(p.positions, 4))
    return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_qk_norm_fwd(const ssd_qk_norm_shape* shape, const void* q, const void* k, const float* w_q,
                    const float* w_k, const float* freq, const int32_t* positions, void* q_out,
                    void* k_out, void* stream) {
  QkDims d{};
  QkPtrs p{q, k, w_q, w_k, freq, positions};
  const int st = qk_check(shape, &d, p);
  if (st != SSD_OK) return st;
  const int o = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (!q_out || !k_out || off(q_out, o) || off(k_out, o)) return SSD_ERR_INVALID_ARG;
  p.q_out = q_out, p.k_out = k_out;
  return qk_run(shape, d, p, false, stream);
}

size_t ssd_qk_norm_workspace_size(const ssd_qk_norm_shape* shape) {
  QkDims d{};
  if (qk_dims(shape, &d) != SSD_OK) return 0;
  return align_up((size_t)bwd_blocks(d) * 2 * d.D * sizeof(float), 256);
}

int ssd_qk_norm_bwd(const ssd_qk_norm_shape* shape, const void* q, const void* k, const float* w_q,
                    const float* w_k, const float* freq, const int32_t* positions,
                    const void* dq_out, const void* dk_out, void* dq, void* dk, float* dw_q,
                    float* dw_k, void* workspace, size_t workspace_bytes, void* stream) {
  QkDims d{};
  QkPtrs p{q, k, w_q, w_k, freq, positions};
  const int st = qk_check(shape, &d, p);
  if (st != SSD_OK) return st;
  const int e = shape->in_dtype == SSD_BF16 ? 2 : 4, o = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (!dq_out || !dk_out || !dq || !dk || off(dq_out, e) || off(dk_out, e) || off(dq, o) ||
      off(dk, o) || !w_q != !dw_q || !w_k != !dw_k || off(dw_q, 4) || off(dw_k, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || off(workspace, 16) || workspace_bytes < ssd_qk_norm_workspace_size(shape))
    return SSD_ERR_WORKSPACE;
  p.dqo = dq_out, p.dko = dk_out, p.dq = dq, p.dk = dk, p.dw_q = dw_q, p.dw_k = dw_k;
  p.part = static_cast<float*>(workspace);
  return qk_run(shape, d, p, true, stream);
}

}  // extern "C"
