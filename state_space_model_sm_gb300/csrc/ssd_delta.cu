// The gated delta rule: the scan whose state is corrected towards each value.
//     delta_t = softplus(dt + dt_bias),  a_t = exp(delta_t A),  b_t = sigmoid(beta)
//     h <- a_t h,   h <- h + b_t (v_t - h k_t) k_t^T,   y_t = scale h q_t
// for a state h (headdim x dstate) of each head.
//
// By chunks of 64 tokens.  With G the running sum of log a inside a chunk, S the state
// in front of it and rows for tokens, the corrections U (64 x headdim) solve
//     (I + M) U = b (V - e^G K S^T),   M[i, j] = b_i e^(G_i - G_j) k_i . k_j   (j < i)
// and then  Y = scale (e^G Q S^T + ((Q K^T) e^(G_i - G_j))_{j <= i} U),
//           S' = e^(G_63) S + (e^(G_63 - G) U)^T K.
// X = (I + M)^-1 does not depend on the state, so the work splits into what every
// chunk does by itself (k_delta_prep: X; k_delta_out: Y) and the chain over the chunks
// (k_delta_chain: U and the states), whose rows p of the state are independent.
//
// Numerics: all matrix products run on the tensor cores with planes of fp32 values
// (warp_mma.cuh).  What reaches a state, a state's gradient or a parameter's gradient is
// three planes of bf16 (X and the pairs' gradients) or two of fp16 with rows scaled (the
// chains), 2^-22 of a value or 2^-39 of its row's largest, so that a token stays good next
// to others of its chunk that are up to 10^6 times larger; what only reaches a bf16 output
// is two planes of bf16, 2^-16 of each value.  Sums and states are fp32.  Log decays are summed and kept as two floats,
// so that a strong decay early in a chunk takes nothing from the differences behind it.
//
// 64 tokens a chunk: X takes 64^2 / 2 products a token, and the chain's length is the
// number of chunks.  tcgen05 is not used: the chain's three dependent products a chunk would
// each go through tensor memory and back, where mma.sync takes the accumulators as its
// next left operand where they are.  The other kernels could stack two products with the
// same right operand to its 128 rows (64 tokens are half its rate); that was not tried.
// mma.sync's rate, measured as 8 clocks an instruction and SM quarter, is what the
// products' bounds below are of.
//
// Times below are, unless said, of a training step's sequences: 4 x 4096 tokens of 24 heads
// in 12 groups, 64 value rows, 128 key columns, bf16, that is 6144 chunks of a head.
#include <cuda_bf16.h>
#include <math.h>

#include "layer_math.cuh"
#include "ssd_internal.h"
#include "tc_ptx.cuh"
#include "warp_mma.cuh"

namespace ssd {
namespace {

using namespace wm;
using lm::cp_async;
using lm::cp_commit;
using lm::cp_wait;
using lm::ex2;
using lm::from_f;
using lm::sigmoid;
using lm::softplus;
using lm::to_f;

constexpr int kC = 64;       // tokens of a chunk
constexpr int kTP = kC + 8;  // pitch of tiles with a chunk's tokens or 64 value rows across
constexpr int kF = 68;       // pitch of fp32 tiles of 64 columns

struct DeltaDims {
  int B, T, H, G, P, N, nc;
  int rep;  // heads of a group
  int Ps;   // value rows in the workspace: P up to a multiple of 16
  int NP;   // key columns in the workspace: 64 or 128
  int ip;   // planes of the images of keys and queries
  int nb;   // head blocks of a group in the gradient
  int no;   // and in the outputs' kernel
  int sms;  // SMs of the device
  int W, cs;  // segments of a sequence in the chains, and chunks of one
  float scale;
  int64_t qs, qb, ks, kb, vs, vb;  // elements between tokens, and between batch rows
  int vq, vk, vv, vdy;             // whether rows can be read 16 bytes at a time
  int wide, wide_k;                // whether pairs of y's or dv's, of dq's and dk's columns can be written at once
};

// Gates of a chunk's tokens: the log2 decays' running sum G in two floats, b, and what
// the chains multiply rows and columns by, with the powers of two that undo the row
// scales of the images of K, Q and X^T (2^k, 2^q, 2^x of each token).
struct Gates {
  float gh[kC], gl[kC], b[kC];
  float fz[kC];  // b e^G 2^k
  float fu[kC];  // e^(G63 - G) 2^k
  float fx[kC];  // 2^x
  float fq[kC];  // scale e^G 2^q (backward)
};
constexpr int kGateCopies = sizeof(Gates) / 16;

struct DeltaWs {
  Gates* gates;  // (B, H, nc)
  bf16* X;       // (B, H, nc, 2, 64, 72) fp16 planes of the transpose of (I + M)^-1
  bf16* K;       // (B, G, nc, planes, 64, NP + 8) fp16 planes of the keys, rows scaled
  bf16* Q;       // the same of the queries (backward)
  float* U;      // (B, H, nc, Ps, 64)  transposed: [p][token]
  float* S0;     // (B, H, nc, Ps, NP)  the state in front of each chunk
  float* ends;  // (B, H, W, Ps, NP)  the state behind each segment from a zero state (W > 1)
  float* move;  // (B, H, W, NP, NP)  and what it makes of the state in front of it
  float* front; // (B, H, W, Ps, NP)  the state in front of each segment
  // backward
  float* Zb;   // (B, H, nc, Ps, 64)  b e^G S k
  float* E;    // (B, H, nc, Ps, 64)  the part of dU from dY
  float* Zd;   // (B, H, nc, Ps, 64)  the part of dU from the state behind the chunk
  float* dR;   // (B, H, nc, Ps, 64)
  float* dS;   // (B, H, nc, Ps, NP)  gradient of the state behind each chunk
  float* part; // (B, H, nc, 2) sums for dA and ddt_bias
  float* dqp;  // (nb, B, T, G, N) head-block parts of dq, dk where nb > 1
  float* dkp;
  size_t total;
};

template <typename T>
constexpr int planes_of() { return sizeof(T) == 2 ? 1 : 3; }

__device__ __forceinline__ int tokens_of(const DeltaDims& d, const int* lengths, int b) {
  if (!lengths) return d.T;
  const int n = lengths[b];
  return n < 0 ? 0 : n > d.T ? d.T : n;
}

__device__ __forceinline__ float decay_between(const Gates& g, int i, int j) {
  return ex2((g.gh[i] - g.gh[j]) + (g.gl[i] - g.gl[j]));
}

// 64 rows of W columns of src as planes of pitch LD; rows from rv and columns from cv
// on are zeros.  vec: rows are 16-byte aligned and cv is a multiple of 16 bytes.
template <typename T, int W, int LD, int THREADS>
__device__ __forceinline__ void load_tile(bf16* dst, const T* src, int64_t ld, int rv, int cv,
                                          bool vec) {
  if constexpr (sizeof(T) == 2) {
    if (vec) {
#pragma unroll 1
      for (int i = threadIdx.x; i < kC * (W / 8); i += THREADS) {
        const int r = i / (W / 8), c = i % (W / 8) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rv && c < cv) v = *reinterpret_cast<const uint4*>(src + r * ld + c);
        *reinterpret_cast<uint4*>(dst + r * LD + c) = v;
      }
    } else {
#pragma unroll 1
      for (int i = threadIdx.x; i < kC * W; i += THREADS) {
        const int r = i / W, c = i % W;
        dst[r * LD + c] = r < rv && c < cv ? src[r * ld + c] : from_f<bf16>(0.f);
      }
    }
  } else {
#pragma unroll 2
    for (int i = threadIdx.x; i < kC * (W / 4); i += THREADS) {
      const int r = i / (W / 4), c = i % (W / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rv) {
        const T* p = src + r * ld + c;
        if (vec) {
          if (c < cv) v = *reinterpret_cast<const float4*>(p);
        } else {
          if (c < cv) v.x = p[0];
          if (c + 1 < cv) v.y = p[1];
          if (c + 2 < cv) v.z = p[2];
          if (c + 3 < cv) v.w = p[3];
        }
      }
      uint32_t a[3], b[3];
      split2<3>(v.x, v.y, a);
      split2<3>(v.z, v.w, b);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint2*>(dst + k * kC * LD + r * LD + c) = make_uint2(a[k], b[k]);
    }
  }
}

// fp32 matrices of the workspace (S0, dS: value rows x key columns; U, Zb, E, Zd, dR:
// value rows x tokens) are held as the accumulators that write them: 16 rows by 8 columns
// after one another, a float4 for each lane, with the lane's two columns of row lane / 4
// and of the row 8 below.  A warp's store or load is then 512 bytes in a row.
__device__ __forceinline__ float4* frag(float* m, int64_t strip, int tiles, int lane) {
  return reinterpret_cast<float4*>(m) + strip * tiles * 32 + lane;
}
__device__ __forceinline__ float4 as4(const float (&c)[4]) {
  return make_float4(c[0], c[1], c[2], c[3]);
}

// 64 value rows (4 strips; zeros from rv rows on) of W columns of the workspace, first
// into registers, all loads in flight, then as NPL planes into a tile of rows.
template <int W, int LD, int THREADS>
struct WsTile {
  static constexpr int kN = kC * (W / 4) / THREADS, kT = W / 8;
  float4 v[kN];
  // the first row and column of this thread's n-th float4
  __device__ __forceinline__ static void at(int n, int* r, int* c) {
    const int i = threadIdx.x + n * THREADS, lane = i & 31;
    *r = i / (32 * kT) * 16 + (lane >> 2), *c = (i >> 5) % kT * 8 + (lane & 3) * 2;
  }
  __device__ __forceinline__ void load(const float* src, int rv) {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int i = threadIdx.x + n * THREADS;
      v[n] = i / (32 * kT) * 16 < rv ? reinterpret_cast<const float4*>(src)[i]
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  template <int NPL>
  __device__ __forceinline__ void store(bf16* dst) const {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      int r, c;
      at(n, &r, &c);
      uint32_t a[NPL], b[NPL];
      split2<NPL>(v[n].x, v[n].y, a);
      split2<NPL>(v[n].z, v[n].w, b);
#pragma unroll
      for (int k = 0; k < NPL; ++k) {
        *reinterpret_cast<uint32_t*>(dst + k * kC * LD + r * LD + c) = a[k];
        *reinterpret_cast<uint32_t*>(dst + k * kC * LD + (r + 8) * LD + c) = b[k];
      }
    }
  }
};

// As load_tile, started asynchronously: bf16 rows with vec.
template <int W, int LD, int THREADS>
__device__ __forceinline__ void copy_tile(bf16* dst, const bf16* src, int64_t ld, int rv, int cv) {
  constexpr int STEP = THREADS / (W / 8);  // rows between a thread's pieces
  const int r0 = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8) * 8;
  const bf16* from = src + r0 * ld + c;
  bf16* to = dst + r0 * LD + c;
#pragma unroll
  for (int r = 0; r < kC; r += STEP, from += STEP * ld, to += STEP * LD) {
    if (r + r0 < rv && c < cv)
      cp_async<16>(to, from);
    else
      *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
  }
}
// A raw tile, asynchronously where it can be (cp_wait and a barrier complete it).
template <typename T, int W, int LD, int THREADS>
__device__ __forceinline__ void fetch_tile(bf16* dst, const T* src, int64_t ld, int rv, int cv,
                                           bool vec) {
  if constexpr (sizeof(T) == 2) {
    if (vec) {
      copy_tile<W, LD, THREADS>(dst, src, ld, rv, cv);
      return;
    }
  }
  load_tile<T, W, LD, THREADS>(dst, src, ld, rv, cv, vec);
}
// Planes of an input's fp16 image.
template <typename T>
constexpr int image_planes() { return sizeof(T) == 2 ? 1 : 2; }

// A raw tile of tokens x 64 value columns, as it is, for reads element by element.
template <typename T>
constexpr int raw_pitch() { return sizeof(T) == 2 ? kTP : kF; }
// Bytes (a multiple of 16) from p on into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

struct Place {  // the (batch, head, chunk) of a block
  int b, h, c;
  int64_t i;  // (b * H + h) * nc + c
};
__device__ __forceinline__ Place place(const DeltaDims& d, unsigned block) {
  Place p;
  const unsigned bh = block / (unsigned)d.nc;
  p.i = block;
  p.c = (int)(block - bh * d.nc);
  p.b = (int)(bh / (unsigned)d.H);
  p.h = (int)(bh - (unsigned)p.b * d.H);
  return p;
}

// ---------------------------------------------------------------------- prep

// Lower part (tiles 0 .. 2 strip + 1) of the 16 rows of strip of K K^T and, with queries,
// of Q K^T over NP columns; tiles of NI planes.
template <int NI, int NP, bool QS>
__device__ __forceinline__ void lower_products(float (&kk)[8][4], float (&qk)[QS ? 8 : 1][4],
                                               const bf16* K, const bf16* Q, int strip, int lane) {
  constexpr int LD = NP + 8;
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      kk[t][e] = 0.f;
      if constexpr (QS) qk[t][e] = 0.f;
    }
#pragma unroll 2
  for (int x = 0; x < NP / 16; ++x) {
    uint32_t a[NI][4], f[NI][4];
#pragma unroll
    for (int p = 0; p < NI; ++p) {
      a_rows<LD>(a[p], K + p * kC * LD, strip * 16, x * 16, lane);
      if constexpr (QS) a_rows<LD>(f[p], Q + p * kC * LD, strip * 16, x * 16, lane);
    }
#pragma unroll
    for (int np = 0; np < 4; ++np)
      if (np <= strip) {
        auto b = [&](int j, uint32_t(&r)[4]) {
          b_rows<LD>(r, K + j * kC * LD, np * 16, x * 16, lane);
        };
        if constexpr (QS)
          mma_planes2<NI, NI, NI, NI, NI>(kk[2 * np], kk[2 * np + 1], a, qk[2 * np], qk[2 * np + 1], f, b);
        else
          mma_planes<NI, NI, NI>(kk[2 * np], kk[2 * np + 1], a, b);
      }
  }
}

constexpr int kPrepThreads = 128;

// Shared memory: the tiles of keys and (backward) queries, whose place the planes of M
// take, and the diagonal blocks in fp32; dY's tile.
template <typename T, int NP, bool BWD>
struct PrepSmem {
  static constexpr size_t tiles = (size_t)planes_of<T>() * kC * (NP + 8) * 2 * (BWD ? 2 : 1);
  static constexpr size_t m = (size_t)3 * kC * kTP * 2, diag = (size_t)4 * 16 * 20 * 4;
  static constexpr size_t one = tiles > m + diag ? tiles : m + diag;
  static constexpr size_t dy = BWD ? (size_t)planes_of<T>() * kC * kTP * 2 : 0;
  static constexpr size_t total = sizeof(Gates) + one + dy;
};

// The scale of row tid / 2 of a tile (two threads a row) and, with `to`, the scaled row as
// fp16 planes.  Returns the inverse.
template <int NI, int NIMG, int NP>
__device__ __forceinline__ float row_image(const bf16* tile, bf16* to) {
  constexpr int LD = NP + 8, W = NP / 2;
  const int r = threadIdx.x >> 1, c0 = (threadIdx.x & 1) * W;
  auto piece = [&](int c, float(&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
#pragma unroll
    for (int l = NI - 1; l >= 0; --l) {
      float x[8];
      lm::unpack<bf16, 8>(lm::ld_raw<bf16, 8>(tile + l * kC * LD + r * LD + c0 + c), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += x[j];
    }
  };
  float m = 0.f;
#pragma unroll 2
  for (int c = 0; c < W; c += 8) {
    float f[8];
    piece(c, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const Scale s = scale_of(m);
  if (to) {
#pragma unroll 2
    for (int c = 0; c < W; c += 8) {
      float f[8];
      piece(c, f);
      uint32_t p[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) split2h(f[2 * j], f[2 * j + 1], s.s, p[j]);
#pragma unroll
      for (int l = 0; l < NIMG; ++l)
        *reinterpret_cast<uint4*>(to + l * kC * LD + r * LD + c0 + c) =
            make_uint4(p[0][l], p[1][l], p[2][l], p[3][l]);
    }
  }
  return s.inv;
}

// Gates, images and X of one chunk of one head; in the backward also
// E^T = dY^T (Q K^T e^(..)).
//
// X^T by strips of 16 columns of X, a warp each: with D_i the inverse of the diagonal
// block i of I + M (by substitution, a column a lane; stable whatever the keys, where a
// run of equal keys makes I + M ill suited to a power series),
//     X_jj = D_j,   X_ij^T = -(sum_{j <= l < i} X_lj^T M_il^T) D_i^T,
// a chain of 16 x 16 products whose left operands are the last accumulators.  Merging
// halves of X by fp32 products from shared memory ran at 88 % of shared memory's rate and
// was slower; what bounds this form is the latency of its dependent steps (substitution,
// then four products deep, then the gates' sums), with four to six blocks an SM to cover it:
// 287 us for a training step's two passes, of which the backward's also has Q K^T and E^T.
// A strip's work differs from the next's, and a warp's place in its block decides its
// scheduler, so strips are turned from block to block (313 us without).  (Several heads a
// block keep K K^T but spill: 261 -> 272 us and more at 16384 chunks.)
template <typename T, int NP, bool BWD>
__global__ void __launch_bounds__(kPrepThreads, sizeof(T) == 2 ? (BWD ? 4 : 6) : 1)
    k_delta_prep(DeltaDims d, const T* __restrict__ q, const T* __restrict__ k,
                 const T* __restrict__ dt, const float* __restrict__ dt_bias,
                 const float* __restrict__ A, const T* __restrict__ beta,
                 const T* __restrict__ dy, const int* __restrict__ lengths, DeltaWs w) {
  constexpr int NI = planes_of<T>(), NIMG = image_planes<T>(), LD = NP + 8;
  using SM = PrepSmem<T, NP, BWD>;
  extern __shared__ __align__(16) unsigned char smem[];
  Gates& g = *reinterpret_cast<Gates*>(smem);
  bf16* const Kt = reinterpret_cast<bf16*>(smem + sizeof(Gates));
  bf16* const Qt = Kt + NI * kC * LD;
  bf16* const yt = reinterpret_cast<bf16*>(smem + sizeof(Gates) + SM::one);
  bf16* const Mp = Kt;
  const int tid = threadIdx.x, lane = tid & 31, strip = ((tid >> 5) + blockIdx.x) & 3;
  float* const diag = reinterpret_cast<float*>(smem + sizeof(Gates) + SM::m) + strip * 16 * 20;
  const Place pl = place(d, blockIdx.x);
  const int n = tokens_of(d, lengths, pl.b), t0 = pl.c * kC;
  if (t0 >= n) return;
  const int rv = min(kC, n - t0), grp = pl.h / d.rep;
  const int64_t ys = (int64_t)d.H * d.P;
  const T* const yg = BWD ? dy + ((int64_t)pl.b * d.T + t0) * ys + (int64_t)pl.h * d.P : nullptr;

  float zt[2] = {0.f, 0.f}, zb[2] = {0.f, 0.f};  // of two tokens a lane of the first warp
  if (strip == 0)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (2 * lane + j < rv) {
        const int64_t at = ((int64_t)pl.b * d.T + t0 + 2 * lane + j) * d.H + pl.h;
        zt[j] = to_f(dt[at]) + (dt_bias ? dt_bias[pl.h] : 0.f);
        zb[j] = to_f(beta[at]);
      }
  fetch_tile<T, NP, LD, kPrepThreads>(Kt, k + pl.b * d.kb + t0 * d.ks + (int64_t)grp * d.N, d.ks, rv,
                                      d.N, d.vk);
  if constexpr (BWD)
    fetch_tile<T, NP, LD, kPrepThreads>(Qt, q + pl.b * d.qb + t0 * d.qs + (int64_t)grp * d.N, d.qs, rv,
                                        d.N, d.vq);
  cp_commit();
  if constexpr (BWD) {
    fetch_tile<T, kC, kTP, kPrepThreads>(yt, yg, ys, rv, d.P, d.vdy);
    cp_commit();
  }
  if (strip == 0) {  // two tokens a lane; sums in two floats, each with its exact rest
    float bb[2], hi[2], lo[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // 2^-150 is 0 in fp32: a bound that changes no decay keeps the sums finite.  By a
      // comparison that is false for NaN, so that a NaN gate stays one
      const float log_a = softplus(zt[j]) * (A[pl.h] * lm::kLog2e);
      hi[j] = 2 * lane + j < rv ? (log_a < -150.f ? -150.f : log_a) : 0.f;
      bb[j] = 2 * lane + j < rv ? sigmoid(zb[j]) : 0.f;
    }
    auto plus = [](float& h, float& l, float h2, float l2) {
      const float t = h + h2, z = t - h, e = (h - (t - z)) + (h2 - z) + (l + l2);
      h = t + e;
      l = e - (h - t);
    };
    plus(hi[1], lo[1], hi[0], lo[0]);
    float rh = hi[1], rl = lo[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float h2 = __shfl_up_sync(0xffffffffu, rh, o), l2 = __shfl_up_sync(0xffffffffu, rl, o);
      if (lane >= o) plus(rh, rl, h2, l2);
    }
    const float bh = __shfl_up_sync(0xffffffffu, rh, 1), bl = __shfl_up_sync(0xffffffffu, rl, 1);
    if (lane > 0) plus(hi[0], lo[0], bh, bl);
    g.gh[2 * lane] = hi[0], g.gl[2 * lane] = lo[0], g.b[2 * lane] = bb[0];
    g.gh[2 * lane + 1] = rh, g.gl[2 * lane + 1] = rl, g.b[2 * lane + 1] = bb[1];
  }
  cp_wait<BWD ? 1 : 0>();
  __syncthreads();

  const int r0 = strip * 16 + (lane >> 2), c0 = (lane & 3) * 2;
  const bool first = pl.h % d.rep == 0;  // writes the images of its group
  const int64_t img = (((int64_t)pl.b * d.G + grp) * d.nc + pl.c) * NIMG * kC * LD;
  const float ki = row_image<NI, NIMG, NP>(Kt, first ? w.K + img : nullptr);
  float qi = 0.f;
  if constexpr (BWD) qi = row_image<NI, NIMG, NP>(Qt, first ? w.Q + img : nullptr);
  if ((tid & 1) == 0) {
    const int i = tid >> 1;
    const float eg = ex2(g.gh[i]);
    g.fz[i] = g.b[i] * eg * ki;
    g.fu[i] = decay_between(g, kC - 1, i) * ki;
    g.fq[i] = d.scale * eg * qi;
  }
  float acc[8][4], qk[BWD ? 8 : 1][4];
  lower_products<NI, NP, BWD>(acc, qk, Kt, Qt, strip, lane);
  __syncthreads();  // the tiles are read
#pragma unroll
  for (int t = 0; t < 8; ++t)
    if (t < 2 * strip + 2)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = r0 + e * 8, j = 8 * t + c0;
        float v[2];
#pragma unroll
        for (int f = 0; f < 2; ++f)
          v[f] = j + f < i ? g.b[i] * decay_between(g, i, j + f) * acc[t][2 * e + f] : 0.f;
        if (t < 2 * strip) {
          uint32_t p[3];
          split2<3>(v[0], v[1], p);
#pragma unroll
          for (int l = 0; l < 3; ++l)
            *reinterpret_cast<uint32_t*>(Mp + l * kC * kTP + i * kTP + j) = p[l];
        } else {
          *reinterpret_cast<float2*>(diag + (i & 15) * 20 + (j & 15)) = make_float2(v[0], v[1]);
        }
      }
  __syncwarp();
  {  // column j of D: the diagonal block is this warp's own
    const int j = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == j ? 1.f : 0.f;
#pragma unroll
      for (int l = 0; l < i; ++l) s = fmaf(-diag[i * 20 + l], x[l], s);
      x[i] = s;
    }
    __syncwarp();
    if (lane < 16)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        diag[i * 20 + j] = x[i];
        uint32_t p[3];
        split2<3>(x[i], 0.f, p);
#pragma unroll
        for (int l = 0; l < 3; ++l)
          reinterpret_cast<uint16_t*>(Mp)[l * kC * kTP + (strip * 16 + i) * kTP + strip * 16 + j] =
              (uint16_t)(p[l] & 0xffffu);
      }
  }
  __syncthreads();
  {
    float x[4][2][4];  // X^T, columns of block row i: rows strip * 16 + lane / 4, + 8
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[i][t][e] = i == strip ? diag[(8 * t + c0 + (e & 1)) * 20 + (lane >> 2) + (e >> 1) * 8] : 0.f;
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (i > strip) {
        float s[2][4] = {};
#pragma unroll
        for (int l = 0; l < i; ++l)
          if (l >= strip) {
            uint32_t a[3][4];
            a_from_acc<3>(a, x[l], 0);
            mma_planes<3, 3, 3>(s[0], s[1], a, [&](int j, uint32_t(&r)[4]) {
              b_rows<kTP>(r, Mp + j * kC * kTP, i * 16, l * 16, lane);
            });
          }
        uint32_t a[3][4];
        a_from_acc<3>(a, s, 0);
        mma_planes<3, 3, 3>(x[i][0], x[i][1], a, [&](int j, uint32_t(&r)[4]) {
          b_rows<kTP>(r, Mp + j * kC * kTP, i * 16, i * 16, lane);
        });
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][t][e] = -x[i][t][e];
      }
    float m0, m1;
    row_max<8>(reinterpret_cast<const float(&)[8][4]>(x), m0, m1);
    const Scale s0 = scale_of(m0), s1 = scale_of(m1);
    if ((lane & 3) == 0) g.fx[r0] = s0.inv, g.fx[r0 + 8] = s1.inv;
    bf16* const xp = w.X + pl.i * (2 * kC * kTP);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t p[2];
          split2h(x[i][t][2 * e], x[i][t][2 * e + 1], e ? s1.s : s0.s, p);
#pragma unroll
          for (int l = 0; l < 2; ++l)
            *reinterpret_cast<uint32_t*>(xp + l * kC * kTP + (r0 + 8 * e) * kTP + i * 16 + 8 * t + c0) =
                p[l];
        }
  }
  __syncthreads();
  if (tid < kGateCopies)
    reinterpret_cast<uint4*>(w.gates + pl.i)[tid] = reinterpret_cast<const uint4*>(&g)[tid];
  if constexpr (BWD) {
    // E^T[p][j] = sum_{i >= j} dy[i][p] scale e^(G_i - G_j) q_i . k_j
    bf16* const at = Mp;  // M's planes are read
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = r0 + e * 8, j = 8 * t + c0;
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int f = 0; f < 2; ++f)
          if (t < 2 * strip + 2 && j + f <= i)
            v[f] = d.scale * decay_between(g, i, j + f) * qk[t][2 * e + f];
        uint32_t p[3];
        split2<3>(v[0], v[1], p);
#pragma unroll
        for (int l = 0; l < 3; ++l)
          *reinterpret_cast<uint32_t*>(at + l * kC * kTP + i * kTP + j) = p[l];
      }
    for (int p0 = 0; p0 < d.Ps; p0 += kC) {
      if (p0 > 0) {
        load_tile<T, kC, kTP, kPrepThreads>(yt, yg + p0, ys, rv, d.P - p0, d.vdy);
      } else {
        cp_wait<0>();
      }
      __syncthreads();
      if (p0 + strip * 16 < d.Ps) {
        float e[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) e[t][x] = 0.f;
#pragma unroll 1
        for (int kb = 0; kb < 4; ++kb) {
          uint32_t a[NI][4];
#pragma unroll
          for (int p = 0; p < NI; ++p) a_cols<kTP>(a[p], yt + p * kC * kTP, strip * 16, kb * 16, lane);
#pragma unroll
          for (int np = 0; np < 4; ++np)
            if (np <= kb) mma_planes<NI, 3, 3>(e[2 * np], e[2 * np + 1], a, [&](int j, uint32_t(&r)[4]) {
              b_cols<kTP>(r, at + j * kC * kTP, np * 16, kb * 16, lane);
            });
        }
        float4* to = frag(w.E, (pl.i * d.Ps + p0) / 16 + strip, 8, lane);
#pragma unroll
        for (int t = 0; t < 8; ++t) to[t * 32] = as4(e[t]);
      }
      __syncthreads();
    }
  }
}

// --------------------------------------------------------------------- chain

constexpr int kChainThreads = 160;

template <typename T, int NP>
constexpr size_t chain_stage() {
  return sizeof(Gates) + (size_t)image_planes<T>() * kC * (NP + 8) * 2 +
         (size_t)kC * raw_pitch<T>() * sizeof(T) + (size_t)2 * kC * kTP * 2;
}

// A state strip (16 rows of a warp, NP columns) from or to rows of N floats.
template <int NP>
__device__ __forceinline__ void load_state(float (&S)[NP / 8][4], const float* src, int rows, int N,
                                           int lane) {
  const int r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
  for (int t = 0; t < NP / 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = r + (e >> 1) * 8, j = 8 * t + c + (e & 1);
      S[t][e] = src && i < rows && j < N ? src[(int64_t)i * N + j] : 0.f;
    }
}
template <int NP>
__device__ __forceinline__ void store_state(float* dst, const float (&S)[NP / 8][4], int rows, int N,
                                            int lane) {
  const int r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
  for (int t = 0; t < NP / 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = r + (e >> 1) * 8, j = 8 * t + c + (e & 1);
      if (i < rows && j < N) dst[(int64_t)i * N + j] = S[t][e];
    }
}

// The value rows (tokens for dY) of a chunk as they are, 64 columns from p0 on, by the
// lanes of one warp: rows of 16 bytes by bulk copies, others element by element; rows
// from rv on are zeros, columns from cv on stay as they were.  Returns the bytes that
// will complete on bar.
template <typename T>
__device__ __forceinline__ uint32_t raw_rows(T* dst, const T* src, int64_t ld, int rv, int cv, bool vec,
                                             uint64_t* bar, int lane) {
  constexpr int RP = raw_pitch<T>();
  cv = min(cv, kC);
  for (int r = max(rv, 0) + lane; r < kC; r += 32)
    for (int c = 0; c < kC; ++c) dst[r * RP + c] = from_f<T>(0.f);
  if (rv < kC) tc::fence_async_smem();  // the zeros, before a later chunk's copies
  if (vec) {
    for (int r = lane; r < rv; r += 32) tc::bulk_g2s(dst + r * RP, src + r * ld, cv * sizeof(T), bar);
    return (uint32_t)(rv * cv * sizeof(T));
  }
  for (int r = 0; r < rv; ++r)
    for (int c = lane; c < cv; c += 32) dst[r * RP + c] = src[r * ld + c];
  return 0;
}

// Stages of a chain: filled by a warp of their own (the fifth), used by a warp for each
// strip, which wait for nothing but their stage.
struct ChainBars {
  uint64_t full[2], empty[2];
  int abort, pad[3];
};
constexpr int kFillWarp = 4;

// A strip's 16 value columns of a raw tile as its rows: the accumulator of the transpose.
template <typename T>
__device__ __forceinline__ void raw_strip(float (&c)[8][4], const T* tile, int strip, int lane) {
  constexpr int RP = raw_pitch<T>();
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t x[4];
      a_cols<RP>(x, tile, strip * 16, kb * 16, lane);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        c[2 * kb + (q >> 1)][(q & 1) * 2] = __uint_as_float(x[q] << 16);
        c[2 * kb + (q >> 1)][(q & 1) * 2 + 1] = __uint_as_float(x[q] & 0xffff0000u);
      }
    }
  } else {
    const T* p = tile + (lane & 3) * 2 * RP + strip * 16 + (lane >> 2);
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[t][e] = p[(8 * t + (e & 1)) * RP + (e >> 1) * 8];
  }
}

// Z^T = S K^T, rows of S scaled.
template <int NI, int NP>
__device__ __forceinline__ void state_times_keys(float (&z)[8][4], const float (&S)[NP / 8][4],
                                                 const bf16* kt, Scale s0, Scale s1, int lane) {
  constexpr int LD = NP + 8;
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) z[t][e] = 0.f;
#pragma unroll
  for (int kk = 0; kk < NP / 16; ++kk) {
    uint32_t a[2][4];
    a_from_acc_h(a, S, kk, s0.s, s1.s);
#pragma unroll
    for (int np = 0; np < 4; ++np)
      mma_planes_h<NI>(z[2 * np], z[2 * np + 1], a, [&](int j, uint32_t(&x)[4]) {
        b_rows<LD>(x, kt + j * kC * LD, np * 16, kk * 16, lane);
      });
  }
}
// S <- keep S + the product of the tokens of c with their rows of the tile.  The products are
// summed from zero, W tiles of columns at a time, and added to the state by one rounded
// operation: an accumulation truncates, and with the state as the accumulator a long-lived
// one lost 3e-7 of itself every chunk (7e-5 over 256).  W 8 in the backward's chain (4: 303
// us for 288), 4 in the forward's, whose registers two blocks an SM share.
template <int NI, int NP, int W = 4>
__device__ __forceinline__ void add_outer(float (&S)[NP / 8][4], float keep, const float (&c)[8][4],
                                          const bf16* kt, Scale s0, Scale s1, int lane) {
  constexpr int LD = NP + 8;
  uint32_t a[4][2][4];
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) a_from_acc_h(a[kb], c, kb, s0.s, s1.s);
#pragma unroll
  for (int n = 0; n < NP / 8; n += W) {
    float t[W][4] = {};
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
      for (int j = NI - 1; j >= 0; --j) {
        uint32_t x[W / 2][4];
#pragma unroll
        for (int h = 0; h < W / 2; ++h)
          b_cols<LD>(x[h], kt + j * kC * LD, n * 8 + h * 16, kb * 16, lane);
#pragma unroll
        for (int i = 1; i >= 0; --i)
          if (i + j < 2)
#pragma unroll
            for (int h = 0; h < W; ++h)
              mma16816h(t[h], a[kb][i], x[h >> 1][(h & 1) * 2], x[h >> 1][(h & 1) * 2 + 1]);
      }
#pragma unroll
    for (int h = 0; h < W; ++h)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const float f = o ? s1.inv : s0.inv;
        const float2 was = make_float2(S[n + h][2 * o], S[n + h][2 * o + 1]);
        const float2 v = __ffma2_rn(make_float2(t[h][2 * o], t[h][2 * o + 1]), make_float2(f, f),
                                    __fmul2_rn(was, make_float2(keep, keep)));
        S[n + h][2 * o] = v.x, S[n + h][2 * o + 1] = v.y;
      }
  }
}
// A strip's rows times f0 and f1.
template <int NT>
__device__ __forceinline__ void scale_rows(float (&c)[NT][4], float f0, float f1) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float2 a = __fmul2_rn(make_float2(c[t][0], c[t][1]), make_float2(f0, f0));
    const float2 b = __fmul2_rn(make_float2(c[t][2], c[t][3]), make_float2(f1, f1));
    c[t][0] = a.x, c[t][1] = a.y, c[t][2] = b.x, c[t][3] = b.y;
  }
}
// Its columns (tokens 8 t + t2, + 1) times the tokens' factors, then its rows times g0 and
// g1: a state's or a gradient's size, which may be any, comes last.
__device__ __forceinline__ void scale_tokens(float (&c)[8][4], const float* f, int t2, float g0, float g1) {
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const float2 x = *reinterpret_cast<const float2*>(f + 8 * t + t2);
    const float2 a = __fmul2_rn(__fmul2_rn(make_float2(c[t][0], c[t][1]), x), make_float2(g0, g0));
    const float2 b = __fmul2_rn(__fmul2_rn(make_float2(c[t][2], c[t][3]), x), make_float2(g1, g1));
    c[t][0] = a.x, c[t][1] = a.y, c[t][2] = b.x, c[t][3] = b.y;
  }
}
template <int NT>
__device__ __forceinline__ void store_strip(float* m, int64_t strip, const float (&c)[NT][4], int lane) {
  float4* p = frag(m, strip, NT, lane);
#pragma unroll
  for (int t = 0; t < NT; ++t) p[t * 32] = as4(c[t]);
}

// A block of a chain: 64 rows (value rows, or rows of a segment's move) of one segment.
struct Piece {
  int b, h, p0, n;        // first row; tokens of the sequence
  int seg, c0, count;     // first chunk, chunks
  int strips;
  bool moving, last, idle;  // rows of the move; holds the sequence's last chunk
  int64_t bh;
};
// (REV: of the backward's chain, whose pass over segments leaves out the first one.)
template <int NP, bool SEG, bool REV>
__device__ __forceinline__ Piece piece(const DeltaDims& d, const int* lengths) {
  Piece p;
  const unsigned vt = (d.Ps + kC - 1) / kC, tiles = SEG ? vt + NP / kC : vt, segs = SEG ? d.W - 1 : d.W;
  const unsigned x = blockIdx.x / tiles, tile = blockIdx.x - x * tiles, bh = x / segs;
  p.seg = (int)(x - bh * segs) + (SEG && REV ? 1 : 0);
  p.bh = bh;
  p.b = (int)(bh / (unsigned)d.H), p.h = (int)(bh - (unsigned)p.b * d.H);
  p.n = tokens_of(d, lengths, p.b);
  const int nc = (p.n + kC - 1) / kC;
  p.c0 = p.seg * d.cs;
  p.count = max(0, min(nc, p.c0 + d.cs) - p.c0);
  p.moving = tile >= vt;
  p.p0 = (int)(p.moving ? tile - vt : tile) * kC;
  p.strips = min(4, ((p.moving ? NP : d.Ps) - p.p0) / 16);
  p.last = p.count > 0 ? p.c0 + p.count == nc : p.seg == 0;
  p.idle = SEG ? p.moving && p.seg == (REV ? d.W - 1 : 0) : p.count == 0 && !p.last;
  return p;
}
// The state that a block starts from: the sequence's first (for the backward: last) one,
// what the join left, or in the pass over segments zeros or the identity's rows.
template <int NP, bool SEG, bool REV>
__device__ __forceinline__ void start_state(float (&S)[NP / 8][4], const DeltaDims& d, const Piece& p,
                                            int row, const float* first, const float* front, int lane) {
  const bool whole = REV ? p.last : p.seg == 0;
  if (!SEG && !whole) {
    load_state<NP>(S, front + ((p.bh * d.W + p.seg) * d.Ps + row) * NP, 16, NP, lane);
  } else if (SEG && (p.moving || !whole)) {
    const int r = row + (lane >> 2), c = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < NP / 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[t][e] = p.moving && 8 * t + c + (e & 1) == r + (e >> 1) * 8 ? 1.f : 0.f;
  } else {
    load_state<NP>(S, first ? first + (p.bh * d.P + row) * d.N : nullptr, d.P - row, d.N, lane);
  }
}
template <int NP, bool SEG>
__device__ __forceinline__ void end_state(const float (&S)[NP / 8][4], const DeltaDims& d, const Piece& p,
                                          int row, float* last, const DeltaWs& w, int lane) {
  if constexpr (SEG) {
    float* to = p.moving ? w.move + ((p.bh * d.W + p.seg) * NP + row) * NP
                         : w.ends + ((p.bh * d.W + p.seg) * d.Ps + row) * NP;
    store_state<NP>(to, S, 16, NP, lane);
  } else if (last) {
    store_state<NP>(last + (p.bh * d.P + row) * d.N, S, d.P - row, d.N, lane);
  }
}

// The state in front of each segment: front_0 is the sequence's first state, front_1 =
// ends_0 (which starts from it), front_j+1 = ends_j + front_j move_j.  16 rows a block;
// four groups of threads take a quarter of the products' sums each.  REV: the gradient
// behind each segment, from the last one's (0: it starts from the sequence's) to the first.
template <int NP, bool REV>
__global__ void __launch_bounds__(4 * NP) k_delta_join(DeltaDims d, DeltaWs w) {
  __shared__ float s[16][NP], part[4][16][NP];
  const int col = threadIdx.x % NP, g = threadIdx.x / NP, strips = d.Ps / 16;
  const int64_t bh = blockIdx.x / strips;
  const int row = (int)(blockIdx.x % strips) * 16;
  for (int j = 1; j < d.W; ++j) {
    const int64_t at = bh * d.W + (REV ? d.W - j : j - 1);
    const float* e = w.ends + (at * d.Ps + row) * NP + col;
    float* f = w.front + ((REV ? at - 1 : at + 1) * d.Ps + row) * NP + col;
    float own[4];  // rows 4 g .. of this column
#pragma unroll
    for (int r = 0; r < 4; ++r) own[r] = e[(4 * g + r) * NP];
    if (j > 1) {
      const float* m = w.move + (at * NP + g * (NP / 4)) * NP + col;
      float b[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) b[r] = 0.f;
#pragma unroll 16
      for (int k = 0; k < NP / 4; ++k) {
        const float x = m[k * NP];
#pragma unroll
        for (int r = 0; r < 16; ++r) b[r] = fmaf(s[r][g * (NP / 4) + k], x, b[r]);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) part[g][r][col] = b[r];
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int p = 0; p < 4; ++p) own[r] += part[p][4 * g + r][col];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) s[4 * g + r][col] = f[(4 * g + r) * NP] = own[r];
    __syncthreads();
  }
}

// The chain over a head's chunks: 64 value rows a block, a strip of 16 rows a warp with
// its state in registers (16 x NP fp32, an accumulator).  A chunk is three products,
//     Z^T = S K^T,   U^T = (b (V - e^G Z))^T X^T,   S <- e^G63 S + (e^(G63 - G) U)^T K,
// each left operand formed from the last accumulator.
// Left operands are two fp16 planes of rows scaled by their largest value, K is one
// (bf16 inputs) and X two: 316 products of 16 x 8 x 16 a chunk, where three planes of
// bf16 take 504.  A warp issues its strip's at 8 clocks each, which bounds a chunk by 1.3 us;
// it takes 3.2 with a block an SM and 5.0 with two, the rest of which is the accumulators'
// way into operands: maxima, scales, planes.  209 us a pass (96 chains of 64 chunks); two
// warps a strip, which exchange halves, were slower.  KEEP: also writes b e^G Z, for the
// backward.  (Two blocks of five warps put three on one quarter of the SM, which holds three of
// 168 registers a thread: the bound that the compiler takes from two blocks of six warps.)
//
// Few heads leave most of the machine idle, so a long sequence is cut into W segments of cs
// chunks.  A chunk's step is linear in the state and the values, row by row: the state
// behind a segment is  ends + front move,  with `ends` from a zero state and `move` the
// rows of the identity taken through the segment without values.  SEG is the pass that
// forms both (no other output); k_delta_join adds them up to each segment's front; the
// pass that writes the states and U then runs all segments at once.
template <typename T, int NP, bool KEEP, bool SEG>
__global__ void __launch_bounds__(192, 2)
    k_delta_chain(DeltaDims d, const T* __restrict__ v, const float* __restrict__ init,
                  const int* __restrict__ lengths, DeltaWs w, float* __restrict__ final_states,
                  int* status) {
  constexpr int NI = image_planes<T>(), LD = NP + 8, RP = raw_pitch<T>();
  extern __shared__ __align__(16) unsigned char smem[];
  ChainBars& sm = *reinterpret_cast<ChainBars*>(smem);
  const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5;
  const Piece pc = piece<NP, SEG, false>(d, lengths);
  const int p0 = pc.p0, b = pc.b, h = pc.h, n = pc.n, c0 = pc.c0, nc = pc.count;
  const int64_t bh = pc.bh;
  if (pc.idle) return;
  const int strips = pc.strips;
  unsigned char* const stages = smem + sizeof(ChainBars);
  constexpr size_t STAGE = chain_stage<T, NP>(), VT = sizeof(Gates) + NI * kC * LD * 2;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.full[i], 32);
      tc::mbar_init(&sm.empty[i], strips);
    }
    tc::fence_mbar_init();
    sm.abort = 0;
  }
  for (int i = threadIdx.x; i < 2 * kC * RP; i += kChainThreads)  // columns that no copy fills
    reinterpret_cast<T*>(stages + (i >= kC * RP ? STAGE : 0) + VT)[i % (kC * RP)] = from_f<T>(0.f);
  tc::fence_async_smem();
  __syncthreads();

  if (strip == kFillWarp) {
    const T* const vg = v + b * d.vb + (int64_t)h * d.P + p0;
    const bf16* const kg = w.K + ((int64_t)b * d.G + h / d.rep) * d.nc * NI * kC * LD;
    int c = 0;
    for (; c < nc; ++c) {
      const int s = c & 1, cc = c0 + c;
      if (!tc::mbar_wait(&sm.empty[s], ((c >> 1) & 1) ^ 1, status, &sm.abort)) break;
      unsigned char* at = stages + s * STAGE;
      uint64_t* bar = &sm.full[s];
      if (lane == 0) {
        tc::bulk_g2s(at, w.gates + bh * d.nc + cc, sizeof(Gates), bar);
        tc::bulk_g2s(at + sizeof(Gates), kg + (int64_t)cc * NI * kC * LD, NI * kC * LD * 2, bar);
        tc::bulk_g2s(at + VT + kC * RP * sizeof(T), w.X + (bh * d.nc + cc) * (2 * kC * kTP),
                     2 * kC * kTP * 2, bar);
      }
      uint32_t raw = 0;
      if (!SEG || !pc.moving)
        raw = raw_rows<T>(reinterpret_cast<T*>(at + VT), vg + (int64_t)cc * kC * d.vs, d.vs,
                          min(kC, n - cc * kC), d.P - p0, d.vv, bar, lane);
      if (lane == 0)
        tc::mbar_arrive_expect_tx(bar, raw + sizeof(Gates) + NI * kC * LD * 2 + 2 * kC * kTP * 2);
      else
        tc::mbar_arrive(bar);
    }
    // what is on its way lands before the block ends (where its strips gave up)
    for (int i = max(0, c - 2); i < c; ++i) tc::mbar_drain(&sm.full[i & 1], (i >> 1) & 1);
    return;
  }
  if (strip >= strips) return;
  const int row = p0 + strip * 16;  // this warp's first value row
  float S[NP / 8][4];
  start_state<NP, SEG, false>(S, d, pc, row, init, w.front, lane);
  const int t2 = (lane & 3) * 2;
  for (int c = 0; c < nc; ++c) {
    const int s = c & 1;
    if (!tc::mbar_wait(&sm.full[s], (c >> 1) & 1, status, &sm.abort)) return;
    const unsigned char* at = stages + s * STAGE;
    const Gates& g = *reinterpret_cast<const Gates*>(at);
    const bf16* kt = reinterpret_cast<const bf16*>(at + sizeof(Gates));
    const T* vt = reinterpret_cast<const T*>(at + VT);
    const bf16* xt = reinterpret_cast<const bf16*>(vt + kC * RP);
    const int64_t srow = ((bh * d.nc + c0 + c) * d.Ps + row) / 16;
    float m0, m1, a0, a1;
    row_max<NP / 8>(S, m0, m1);
    const Scale s0 = scale_of(m0), s1 = scale_of(m1);
    float r[8][4];
    state_times_keys<NI, NP>(r, S, kt, s0, s1, lane);
    if constexpr (!SEG) store_strip<NP / 8>(w.S0, srow, S, lane);
    // r = b (v - e^G z) 2^x, of the value rows g8 and g8 + 8 and tokens 8 t + t2, + 1
    scale_tokens(r, g.fz, t2, s0.inv, s1.inv);
    if constexpr (KEEP && !SEG) store_strip<8>(w.Zb, srow, r, lane);
    float u[8][4];
    raw_strip<T>(u, vt, strip, lane);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float2 bi = *reinterpret_cast<const float2*>(g.b + 8 * t + t2);
      const float2 fx = *reinterpret_cast<const float2*>(g.fx + 8 * t + t2);
      const float2 m1 = make_float2(-1.f, -1.f);
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const float2 v = __fmul2_rn(bi, make_float2(u[t][2 * o], u[t][2 * o + 1]));
        const float2 x = __fmul2_rn(fx, __ffma2_rn(make_float2(r[t][2 * o], r[t][2 * o + 1]), m1, v));
        r[t][2 * o] = x.x, r[t][2 * o + 1] = x.y;
      }
    }
    row_max<8>(r, a0, a1);
    const Scale q0 = scale_of(a0), q1 = scale_of(a1);
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) u[t][e] = 0.f;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t a[2][4];
      a_from_acc_h(a, r, kb, q0.s, q1.s);
#pragma unroll
      for (int np = kb; np < 4; ++np)
        mma_planes_h<2>(u[2 * np], u[2 * np + 1], a, [&](int j, uint32_t(&x)[4]) {
          b_cols<kTP>(x, xt + j * kC * kTP, np * 16, kb * 16, lane);
        });
    }
    scale_rows(u, q0.inv, q1.inv);
    if constexpr (!SEG) store_strip<8>(w.U, srow, u, lane);
    scale_tokens(u, g.fu, t2, 1.f, 1.f);
    row_max<8>(u, a0, a1);
    add_outer<NI, NP>(S, ex2(g.gh[kC - 1]), u, kt, scale_of(a0), scale_of(a1), lane);
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.empty[s]);
  }
  end_state<NP, SEG>(S, d, pc, row, pc.last ? final_states : nullptr, w, lane);
}

template <typename T, int NP>
constexpr size_t chain_smem() { return sizeof(ChainBars) + 2 * chain_stage<T, NP>(); }

// ----------------------------------------------------------------------- out

constexpr int kOutThreads = 256;

// Planes of values that only reach an output of type TO.
template <typename TO>
constexpr int out_planes() { return sizeof(TO) == 2 ? 2 : 3; }

// Shared memory: queries; keys, whose place the state's planes take; U; the pairs.
template <typename T, typename TO, int NP>
struct OutSmem {
  static constexpr size_t raw = (size_t)planes_of<T>() * kC * (NP + 8) * 2;
  static constexpr size_t st = (size_t)out_planes<TO>() * kC * (NP + 8) * 2;
  static constexpr size_t one = raw > st ? raw : st;
  static constexpr size_t tok = (size_t)out_planes<TO>() * kC * kTP * 2;
  static constexpr size_t total = sizeof(Gates) + raw + one + 2 * tok;
};

// Y of one chunk of the heads of one head block: 16 tokens by half of 64 value columns a
// warp, in passes of 64 value columns of a head.  Q K^T is formed once for the heads, by
// halves of the tokens; a head's decays make its planes of it.  The next pass's states and
// corrections are on their way under a pass's products.  Bound by shared memory (the
// states' planes are read by four warps; by two, with 32 tokens by 16 columns a warp, it
// spills: 295 -> 346 us for 16384 chunks) and the work around the products: 134 us, of
// which reading states and corrections and writing y would take 48 at the copy rate.
// Outputs formed in the chain, with operands of 11 bits, saved an eighth of a prompt but
// were off by 2^-12 of the largest y.
template <typename T, typename TO, int NP>
__global__ void __launch_bounds__(kOutThreads, sizeof(T) == 2 && sizeof(TO) == 2 ? 2 : 1)
    k_delta_out(DeltaDims d, const T* __restrict__ q, const T* __restrict__ k,
                const int* __restrict__ lengths, DeltaWs w, TO* __restrict__ y) {
  constexpr int NI = planes_of<T>(), NL = out_planes<TO>(), LD = NP + 8;
  using SM = OutSmem<T, TO, NP>;
  extern __shared__ __align__(16) unsigned char smem[];
  Gates& g = *reinterpret_cast<Gates*>(smem);
  bf16* const qt = reinterpret_cast<bf16*>(smem + sizeof(Gates));
  bf16* const kt = qt + SM::raw / 2;  // and the state's planes after the keys'
  bf16* const ut = kt + SM::one / 2;
  bf16* const pt = ut + SM::tok / 2;
  // (strips have products with up to their own block of tokens: each scheduler gets a long
  // and a short one)
  const int tid = threadIdx.x, lane = tid & 31, half = tid >> 7;
  const int strip = half ? 3 - ((tid >> 5) & 3) : tid >> 5;
  const unsigned b1 = blockIdx.x / d.nc, b2 = b1 / d.no;
  const int c = (int)(blockIdx.x - b1 * d.nc), hb = (int)(b1 - b2 * d.no);
  const int b = (int)(b2 / d.G), grp = (int)(b2 - (unsigned)b * d.G);
  const int h0 = grp * d.rep + (int)((unsigned)d.rep * hb / d.no);
  const int h1 = grp * d.rep + (int)((unsigned)d.rep * (hb + 1) / d.no);
  const int n = tokens_of(d, lengths, b), t0 = c * kC;
  const int rows = min(kC, d.T - t0);  // of the output; tokens from n on are padding
  const int64_t ys = (int64_t)d.H * d.P;
  TO* const yb = y + ((int64_t)b * d.T + t0) * ys;
  if (t0 >= n) {
    const int cols = (h1 - h0) * d.P;
#pragma unroll 1
    for (int i = tid; i < rows * cols; i += kOutThreads)
      yb[i / cols * ys + (int64_t)h0 * d.P + i % cols] = from_f<TO>(0.f);
    return;
  }
  const int rv = min(kC, n - t0);
  fetch_tile<T, NP, LD, kOutThreads>(qt, q + b * d.qb + t0 * d.qs + (int64_t)grp * d.N, d.qs, rv, d.N,
                                     d.vq);
  fetch_tile<T, NP, LD, kOutThreads>(kt, k + b * d.kb + t0 * d.ks + (int64_t)grp * d.N, d.ks, rv, d.N,
                                     d.vk);
  cp_commit();
  WsTile<NP, LD, kOutThreads> ws;
  WsTile<kC, kTP, kOutThreads> wu;
  uint4 gates = make_uint4(0, 0, 0, 0);
  auto ahead = [&](int h, int p0) {
    const int64_t at = ((int64_t)b * d.H + h) * d.nc + c;
    ws.load(w.S0 + (at * d.Ps + p0) * NP, min(kC, d.Ps - p0));
    wu.load(w.U + (at * d.Ps + p0) * kC, min(kC, d.Ps - p0));
    if (p0 == 0 && tid < kGateCopies) gates = reinterpret_cast<const uint4*>(w.gates + at)[tid];
  };
  ahead(h0, 0);
  cp_wait<0>();
  __syncthreads();
  const int r0 = strip * 16 + (lane >> 2), c0 = (lane & 3) * 2;
  float s[4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
  if (2 * half <= strip)
#pragma unroll 2
    for (int kk = 0; kk < NP / 16; ++kk) {
      uint32_t a[NI][4];
#pragma unroll
      for (int p = 0; p < NI; ++p) a_rows<LD>(a[p], qt + p * kC * LD, strip * 16, kk * 16, lane);
#pragma unroll
      for (int np = 0; np < 2; ++np)
        mma_planes<NI, NI, NI>(s[2 * np], s[2 * np + 1], a, [&](int j, uint32_t(&x)[4]) {
          b_rows<LD>(x, kt + j * kC * LD, half * 32 + np * 16, kk * 16, lane);
        });
    }
  for (int h = h0; h < h1; ++h) {
    float f0 = 0.f, f1 = 0.f;
    for (int p0 = 0; p0 < d.Ps; p0 += kC) {
      __syncthreads();  // the last pass's tiles (at first: the keys) are read
      ws.template store<NL>(kt);
      wu.template store<NL>(ut);
      if (p0 == 0 && tid < kGateCopies) reinterpret_cast<uint4*>(&g)[tid] = gates;
      __syncthreads();
      if (p0 + kC < d.Ps) ahead(h, p0 + kC);
      else if (h + 1 < h1) ahead(h + 1, 0);
      if (p0 == 0) {  // the head's pairs
        f0 = d.scale * ex2(g.gh[r0]), f1 = d.scale * ex2(g.gh[r0 + 8]);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = r0 + e * 8, j = half * 32 + 8 * t + c0;
            float v[2];
#pragma unroll
            for (int f = 0; f < 2; ++f)
              v[f] = j + f <= i ? d.scale * decay_between(g, i, j + f) * s[t][2 * e + f] : 0.f;
            uint32_t x[NL];
            split2<NL>(v[0], v[1], x);
#pragma unroll
            for (int l = 0; l < NL; ++l)
              *reinterpret_cast<uint32_t*>(pt + l * kC * kTP + i * kTP + j) = x[l];
          }
        __syncthreads();
      }
      if (p0 + half * 32 >= d.Ps) continue;
      float o[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
#pragma unroll 2
      for (int kk = 0; kk < NP / 16; ++kk) {
        uint32_t a[NI][4];
#pragma unroll
        for (int p = 0; p < NI; ++p) a_rows<LD>(a[p], qt + p * kC * LD, strip * 16, kk * 16, lane);
#pragma unroll
        for (int np = 0; np < 2; ++np)
          mma_planes<NI, NL, max2(NI, NL)>(o[2 * np], o[2 * np + 1], a, [&](int j, uint32_t(&x)[4]) {
            b_rows<LD>(x, kt + j * kC * LD, half * 32 + np * 16, kk * 16, lane);
          });
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t][0] *= f0, o[t][1] *= f0, o[t][2] *= f1, o[t][3] *= f1;
#pragma unroll 1
      for (int kb = 0; kb <= strip; ++kb) {
        uint32_t a[NL][4];
#pragma unroll
        for (int l = 0; l < NL; ++l) a_rows<kTP>(a[l], pt + l * kC * kTP, strip * 16, kb * 16, lane);
#pragma unroll
        for (int np = 0; np < 2; ++np)
          mma_planes<NL, NL, NL>(o[2 * np], o[2 * np + 1], a, [&](int j, uint32_t(&x)[4]) {
            b_rows<kTP>(x, ut + j * kC * kTP, half * 32 + np * 16, kb * 16, lane);
          });
      }
      TO* const yo = yb + (int64_t)h * d.P;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = r0 + e * 8, p = p0 + half * 32 + 8 * t + c0;
          if (i < rows && p < d.P) {
            const bool in = i < rv;
            lm::st_two(yo + i * ys + p,
                       make_float2(in ? o[t][2 * e] : 0.f, in ? o[t][2 * e + 1] : 0.f), p + 1 < d.P,
                       d.wide);
          }
        }
    }
  }
}

// ---------------------------------------------------------------------- back

template <typename T, int NP>
constexpr size_t back_stage() {
  return chain_stage<T, NP>() + (size_t)image_planes<T>() * kC * (NP + 8) * 2;
}
template <typename T, int NP>
constexpr size_t back_smem() { return sizeof(ChainBars) + 2 * back_stage<T, NP>(); }

// The chain of the backward, from the last chunk to the first, with the gradient of the
// state behind the chunk in registers:
//     dU^T = E^T + (dS K^T) e^(G63 - G),   dR^T = dU^T X,
//     dS <- e^G63 dS - (b e^G dR)^T K + (scale e^G dY)^T Q,
// in the manner of k_delta_chain: 444 products a chunk, 288 us (96 chains of 64 chunks,
// 4.5 us each).  dR's part is added before dY's rows are taken up: both at once would be
// 178 registers with 64 key columns, and a block an SM where two fit (144).
template <typename T, int NP, bool SEG>
__global__ void __launch_bounds__(kChainThreads)
    k_delta_back(DeltaDims d, const T* __restrict__ dy, const float* __restrict__ dfinal,
                 const int* __restrict__ lengths, DeltaWs w, float* __restrict__ dinit, int* status) {
  constexpr int NI = image_planes<T>(), LD = NP + 8, RP = raw_pitch<T>();
  extern __shared__ __align__(16) unsigned char smem[];
  ChainBars& sm = *reinterpret_cast<ChainBars*>(smem);
  const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5;
  const Piece pc = piece<NP, SEG, true>(d, lengths);
  const int p0 = pc.p0, b = pc.b, h = pc.h, n = pc.n, nc = pc.count, end = pc.c0 + pc.count - 1;
  const int64_t bh = pc.bh;
  if (pc.idle) return;
  const int strips = pc.strips;
  unsigned char* const stages = smem + sizeof(ChainBars);
  constexpr size_t STAGE = back_stage<T, NP>(), IMG = NI * kC * LD * 2;
  constexpr size_t YT = sizeof(Gates) + 2 * IMG;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.full[i], 32);
      tc::mbar_init(&sm.empty[i], strips);
    }
    tc::fence_mbar_init();
    sm.abort = 0;
  }
  for (int i = threadIdx.x; i < 2 * kC * RP; i += kChainThreads)
    reinterpret_cast<T*>(stages + (i >= kC * RP ? STAGE : 0) + YT)[i % (kC * RP)] = from_f<T>(0.f);
  tc::fence_async_smem();
  __syncthreads();

  if (strip == kFillWarp) {
    const int64_t ys = (int64_t)d.H * d.P;
    const T* const yg = dy + b * (int64_t)d.T * ys + (int64_t)h * d.P + p0;
    const int64_t img = ((int64_t)b * d.G + h / d.rep) * d.nc * NI * kC * LD;
    int i = 0;  // chunks filled, the last one first
    for (; i < nc; ++i) {
      const int s = i & 1, c = end - i;
      if (!tc::mbar_wait(&sm.empty[s], ((i >> 1) & 1) ^ 1, status, &sm.abort)) break;
      unsigned char* at = stages + s * STAGE;
      uint64_t* bar = &sm.full[s];
      if (lane == 0) {
        tc::bulk_g2s(at, w.gates + bh * d.nc + c, sizeof(Gates), bar);
        tc::bulk_g2s(at + sizeof(Gates), w.K + img + (int64_t)c * NI * kC * LD, IMG, bar);
        tc::bulk_g2s(at + sizeof(Gates) + IMG, w.Q + img + (int64_t)c * NI * kC * LD, IMG, bar);
        tc::bulk_g2s(at + YT + kC * RP * sizeof(T), w.X + (bh * d.nc + c) * (2 * kC * kTP),
                     2 * kC * kTP * 2, bar);
      }
      uint32_t raw = 0;
      if (!SEG || !pc.moving)
        raw = raw_rows<T>(reinterpret_cast<T*>(at + YT), yg + (int64_t)c * kC * ys, ys,
                          min(kC, n - c * kC), d.P - p0, d.vdy, bar, lane);
      if (lane == 0)
        tc::mbar_arrive_expect_tx(bar, raw + sizeof(Gates) + 2 * IMG + 2 * kC * kTP * 2);
      else
        tc::mbar_arrive(bar);
    }
    for (int j = max(0, i - 2); j < i; ++j) tc::mbar_drain(&sm.full[j & 1], (j >> 1) & 1);
    return;
  }
  if (strip >= strips) return;
  const int row = p0 + strip * 16;
  float S[NP / 8][4];
  start_state<NP, SEG, true>(S, d, pc, row, dfinal, w.front, lane);
  const int t2 = (lane & 3) * 2;
  for (int i = 0; i < nc; ++i) {
    const int s = i & 1, c = end - i;
    if (!tc::mbar_wait(&sm.full[s], (i >> 1) & 1, status, &sm.abort)) return;
    const unsigned char* at = stages + s * STAGE;
    const Gates& g = *reinterpret_cast<const Gates*>(at);
    const bf16* kt = reinterpret_cast<const bf16*>(at + sizeof(Gates));
    const bf16* qt = reinterpret_cast<const bf16*>(at + sizeof(Gates) + IMG);
    const T* yt = reinterpret_cast<const T*>(at + YT);
    const bf16* xt = reinterpret_cast<const bf16*>(yt + kC * RP);
    const int64_t srow = ((bh * d.nc + c) * d.Ps + row) / 16;
    float m0, m1, a0, a1;
    row_max<NP / 8>(S, m0, m1);
    const Scale s0 = scale_of(m0), s1 = scale_of(m1);
    float r[8][4];
    state_times_keys<NI, NP>(r, S, kt, s0, s1, lane);
    if constexpr (!SEG) store_strip<NP / 8>(w.dS, srow, S, lane);
    scale_tokens(r, g.fu, t2, s0.inv, s1.inv);
    if constexpr (!SEG) store_strip<8>(w.Zd, srow, r, lane);
    if (!SEG || !pc.moving)
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float4 e = frag(w.E, srow, 8, lane)[t * 32];
      r[t][0] += e.x, r[t][1] += e.y, r[t][2] += e.z, r[t][3] += e.w;
    }
    row_max<8>(r, a0, a1);
    const Scale q0 = scale_of(a0), q1 = scale_of(a1);
    float u[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) u[t][e] = 0.f;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {  // dR^T[p][j] = sum_{i >= j} dU^T[p][i] X[i][j]
      uint32_t a[2][4];
      a_from_acc_h(a, r, kb, q0.s, q1.s);
#pragma unroll
      for (int np = 0; np <= kb; ++np)
        mma_planes_h<2>(u[2 * np], u[2 * np + 1], a, [&](int j, uint32_t(&x)[4]) {
          b_rows<kTP>(x, xt + j * kC * kTP, np * 16, kb * 16, lane);
        });
    }
    scale_tokens(u, g.fx, t2, q0.inv, q1.inv);
    if constexpr (!SEG) store_strip<8>(w.dR, srow, u, lane);
    scale_tokens(u, g.fz, t2, -1.f, -1.f);  // -b e^G dR^T 2^k
    row_max<8>(u, a0, a1);
    add_outer<NI, NP, 8>(S, ex2(g.gh[kC - 1]), u, kt, scale_of(a0), scale_of(a1), lane);
    raw_strip<T>(r, yt, strip, lane);
    scale_tokens(r, g.fq, t2, 1.f, 1.f);  // scale e^G dY^T 2^q
    row_max<8>(r, a0, a1);
    add_outer<NI, NP, 8>(S, 1.f, r, qt, scale_of(a0), scale_of(a1), lane);
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.empty[s]);
  }
  end_state<NP, SEG>(S, d, pc, row, pc.seg == 0 ? dinit : nullptr, w, lane);
}

// ---------------------------------------------------------------------- grad

constexpr int kGradThreads = 512;

// Sums over the tokens of a chunk that the gates' gradients are made of.
struct GradSums {
  float row[4][kC];       // rows of dAqk Aqk - W M, a column block each
  float col[4][kC];       // columns of the same, a row strip each
  float qd[4][kC];        // scale e^G q . (dY S0), a quarter of the key columns each
  float part[2][3][kC];   // U . Zd, dR . Zb, dR . U, half of the value rows each
  float dot[16];          // <dS, S0>, a warp each
};

// Shared memory: dY, dR, U and S0 (then dS) of a tile of value rows; P1 and P2 over
// dR and U; Q and K beside them, or over dY, where they are three planes wide.
template <typename T, typename TO, int NP>
struct GradSmem {
  static constexpr size_t row = kC * (NP + 8) * 2, tok = kC * kTP * 2, ni = planes_of<T>();
  static constexpr bool beside = ni == 1;
  static constexpr size_t values = ni * tok + 6 * tok + 3 * row, qk = 2 * ni * row;
  static constexpr size_t pairs = 2 * out_planes<TO>() * tok;
  static constexpr size_t over = qk + pairs > values ? qk + pairs : values;
  static constexpr size_t head = sizeof(Gates) + sizeof(GradSums);
  static constexpr size_t total = head + (beside ? values + qk : over);
};

// dq, dk, dv, ddt and dbeta of one chunk of the heads of one head block.  Sixteen warps:
// 16 tokens by a quarter of the key columns (or 16 of the chunk's tokens) each.  With
// dAqk = dY U^T (j <= i) and W = dR U^T (j < i),
//     dq = scale e^G dY S0 + P1 K,                       P1 = scale e^(G_i - G_j) dAqk
//     dk = e^(G63 - G) U dS - b e^G dR S0 + P1^T Q + (P2 + P2^T) K,
//                                                        P2 = -b_i e^(G_i - G_j) W
//     dv = b dR,   dbeta = (1 - b) dR . U   (as b_i dL/db_i = W_ii)
// and the gradient of G_i is the row sum less the column sum of dAqk Aqk - W M, plus
// scale e^G q . (dY S0) - dR . (b e^G S0 k) - U . (e^(G63 - G) dS k), where what the
// last token's G takes from the state behind the chunk is added.  Row and column sums are
// of the same products, each sum rounded by itself: 2^-24 of their terms is left of what
// cancels in their difference, which a step whose decay is 0 does not pass on (gates_of).
// Twelve products of 64 x 64 x 64 to 128 a tile of value rows, whose operands each become
// planes in shared memory first: 700 us, 32 thousand clocks a head and chunk of an SM where
// the products alone take 11.  Issue slots are 40 % used, the tensor cores 28 %; a second
// block does not fit (shared memory), and fetching the next head's tiles into registers
// spills.
template <typename T, typename TO, int NP>
__global__ void __launch_bounds__(kGradThreads, 1)
    k_delta_grad(DeltaDims d, const T* __restrict__ q, const T* __restrict__ k,
                 const T* __restrict__ dt, const float* __restrict__ dt_bias,
                 const float* __restrict__ A, const T* __restrict__ dy,
                 const int* __restrict__ lengths, DeltaWs w, TO* __restrict__ dq,
                 TO* __restrict__ dk, TO* __restrict__ dv, TO* __restrict__ ddt,
                 TO* __restrict__ dbeta) {
  constexpr int NI = planes_of<T>(), NL = out_planes<TO>(), LD = NP + 8;
  constexpr int WC = NP / 4, HT = WC / 8;  // key columns and tiles of a warp
  using SM = GradSmem<T, TO, NP>;
  extern __shared__ __align__(16) unsigned char smem[];
  Gates& g = *reinterpret_cast<Gates*>(smem);
  GradSums& sm = *reinterpret_cast<GradSums*>(smem + sizeof(Gates));
  bf16* const base = reinterpret_cast<bf16*>(smem + SM::head);
  bf16* const yt = base;                // dY [token][p]
  bf16* const rt = yt + NI * kC * kTP;  // dR [p][token]
  bf16* const ut = rt + 3 * kC * kTP;   // U [p][token]
  bf16* const st = ut + 3 * kC * kTP;   // S0, then dS [p][n]
  bf16* const qt = SM::beside ? st + 3 * kC * LD : base;
  bf16* const kt = qt + NI * kC * LD;
  bf16* const p1 = SM::beside ? rt : kt + NI * kC * LD;
  bf16* const p2 = p1 + NL * kC * kTP;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, strip = warp & 3, part = warp >> 2;
  const unsigned b1 = blockIdx.x / d.nc, b2 = b1 / d.nb;
  const int c = (int)(blockIdx.x - b1 * d.nc), hb = (int)(b1 - b2 * d.nb);
  const int b = (int)(b2 / d.G), grp = (int)(b2 - (unsigned)b * d.G);
  const int n = tokens_of(d, lengths, b), t0 = c * kC, rows = min(kC, d.T - t0);
  const int rv = max(0, min(kC, n - t0));
  const int h0 = grp * d.rep + (int)((unsigned)d.rep * hb / d.nb);
  const int h1 = grp * d.rep + (int)((unsigned)d.rep * (hb + 1) / d.nb);
  const int r0 = strip * 16 + (lane >> 2), c0 = (lane & 3) * 2;
  const int64_t ys = (int64_t)d.H * d.P, tok = (int64_t)b * d.T + t0;
  const T* const qg = q + b * d.qb + t0 * d.qs + (int64_t)grp * d.N;
  const T* const kg = k + b * d.kb + t0 * d.ks + (int64_t)grp * d.N;

  float tq[HT][4], tk[HT][4];  // dq, dk over the heads: columns part * WC + 8 t + c0
#pragma unroll
  for (int t = 0; t < HT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) tq[t][e] = tk[t][e] = 0.f;
  if (SM::beside && rv > 0) {
    fetch_tile<T, NP, LD, kGradThreads>(qt, qg, d.qs, rv, d.N, d.vq);
    fetch_tile<T, NP, LD, kGradThreads>(kt, kg, d.ks, rv, d.N, d.vk);
    cp_commit();
  }

  if (rv == 0) {  // padding only
    for (int h = h0; h < h1; ++h) {
#pragma unroll 1
      for (int i = tid; i < rows * d.P; i += kGradThreads)
        dv[(tok + i / d.P) * ys + (int64_t)h * d.P + i % d.P] = from_f<TO>(0.f);
      if (tid < rows) {
        ddt[(tok + tid) * d.H + h] = from_f<TO>(0.f);
        dbeta[(tok + tid) * d.H + h] = from_f<TO>(0.f);
      }
      if (tid < 2) w.part[(((int64_t)b * d.H + h) * d.nc + c) * 2 + tid] = 0.f;
    }
  }
  // the next tile's values are fetched into L2 while this one's products run: of this
  // head, of the block's next head, or of the first head of the block that is likely next
  auto ahead = [&](int64_t at, int p0) {
    if (tid >= 6) return;
    const size_t pt = (size_t)(at * d.Ps + p0);
    const int cols = tid < 2 ? NP : kC;
    const float* from = tid == 0 ? w.S0 : tid == 1 ? w.dS : tid == 2 ? w.dR : tid == 3 ? w.U : tid == 4 ? w.Zd : w.Zb;
    prefetch_l2(from + pt * cols, min(kC, d.Ps - p0) * cols * 4);
  };
  auto ahead_of = [&](int h, int p0) {
    if (p0 + kC < d.Ps) {
      ahead(((int64_t)b * d.H + h) * d.nc + c, p0 + kC);
    } else if (h + 1 < h1) {
      ahead(((int64_t)b * d.H + h + 1) * d.nc + c, 0);
    } else if (blockIdx.x + d.sms < gridDim.x) {
      const unsigned i = blockIdx.x + d.sms, j = i / d.nc, k = j / d.nb, l = k / d.G;
      const int h2 = (int)(k - l * d.G) * d.rep + (int)(d.rep * (j - k * d.nb) / d.nb);
      ahead(((int64_t)l * d.H + h2) * d.nc + (i - j * d.nc), 0);
    }
  };

  // the gates' gradients of a head, by the first warp, two tokens a lane: from the sums that
  // the head left, while the next head's first values are on their way
  bool due = false;
  float zd[2], bd[2], ed = 0.f;
  auto gates_of = [&](int h) {
    const int64_t at = ((int64_t)b * d.H + h) * d.nc + c;
    float dg[2], wii[2], last = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = 2 * lane + x;
      float u = 0.f, r = 0.f, ww = 0.f, rs = 0.f, cs = 0.f, qs = 0.f;
#pragma unroll
      for (int p = 0; p < 2; ++p) u += sm.part[p][0][i], r += sm.part[p][1][i], ww += sm.part[p][2][i];
#pragma unroll
      for (int p = 0; p < 4; ++p) rs += sm.row[p][i], cs += sm.col[p][i], qs += sm.qd[p][i];
      dg[x] = (rs - cs) + (qs - r) - u;
      wii[x] = ww;
      last += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) last += __shfl_xor_sync(0xffffffffu, last, o);
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < 16; ++p) ss += sm.dot[p];
    last += ed * ss;
    if (lane == 31) dg[1] += last;
    // sums from each token on
    dg[0] += dg[1];
    float run = dg[0];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float dn = __shfl_down_sync(0xffffffffu, run, o);
      if (lane + o < 32) run += dn;
    }
    const float after = run - dg[0];
    float sa = 0.f, sb = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = 2 * lane + x;
      const float v = dg[x] + after;
      const int64_t o = (tok + i) * d.H + h;
      if (i < rv) {
        // a decay that is 0 in fp32 (ex2 of less than -126) does not move with its gate; the
        // difference of sums leaves their rounding there, and a step has no bound
        const float delta = softplus(zd[x]);
        const bool gone = delta * (A[h] * lm::kLog2e) < -126.f && v == v;
        const float dz = gone ? 0.f : v * A[h] * sigmoid(zd[x]);
        if (!gone) sa = fmaf(v, delta, sa);
        sb += dz;
        ddt[o] = from_f<TO>(dz);
        dbeta[o] = from_f<TO>((1.f - bd[x]) * wii[x]);
      } else if (i < rows) {
        ddt[o] = from_f<TO>(0.f);
        dbeta[o] = from_f<TO>(0.f);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sa += __shfl_xor_sync(0xffffffffu, sa, o);
      sb += __shfl_xor_sync(0xffffffffu, sb, o);
    }
    if (lane == 0) w.part[at * 2] = sa, w.part[at * 2 + 1] = sb;
  };

  for (int h = h0; h < h1 && rv > 0; ++h) {
    const int64_t at = ((int64_t)b * d.H + h) * d.nc + c;
    // the gates' inputs of the two tokens of a lane of the first warp, for the head's end
    float zt[2] = {0.f, 0.f};
    if (warp == 0)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (2 * lane + x < rv)
          zt[x] = to_f(dt[(tok + 2 * lane + x) * d.H + h]) + (dt_bias ? dt_bias[h] : 0.f);
    float da[2][4], wm[2][4], dqh[HT][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) da[t][e] = wm[t][e] = 0.f;
#pragma unroll
    for (int t = 0; t < HT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) dqh[t][e] = 0.f;
    float2 su = make_float2(0.f, 0.f), sr = su, sw = su;  // of two tokens, the same in every load
    float dot = 0.f;
    for (int p0 = 0; p0 < d.Ps; p0 += kC) {
      const int pr = min(kC, d.Ps - p0);
      WsTile<NP, LD, kGradThreads> ws;
      WsTile<kC, kTP, kGradThreads> wr, wu, wz, wb;
      const size_t pt = (size_t)(at * d.Ps + p0);
      ws.load(w.S0 + pt * NP, pr);
      wr.load(w.dR + pt * kC, pr);
      wu.load(w.U + pt * kC, pr);
      wz.load(w.Zd + pt * kC, pr);
      wb.load(w.Zb + pt * kC, pr);
      if (due) {
        gates_of(h - 1);
        due = false;
      }
      __syncthreads();  // the tiles (and, at a head's start, the gates and sums) are read
      fetch_tile<T, kC, kTP, kGradThreads>(yt, dy + tok * ys + (int64_t)h * d.P + p0, ys, rv, d.P - p0,
                                           d.vdy);
      if (p0 == 0 && tid < kGateCopies)
        cp_async<16>(reinterpret_cast<uint4*>(&g) + tid, reinterpret_cast<const uint4*>(w.gates + at) + tid);
      cp_commit();
      ws.template store<3>(st);
      wr.template store<3>(rt);
      wu.template store<3>(ut);
#pragma unroll
      for (int i = 0; i < wr.kN; ++i) {
        const float4 r = wr.v[i], u = wu.v[i], z = wz.v[i], x = wb.v[i];
        su.x = fmaf(u.x, z.x, fmaf(u.z, z.z, su.x)), su.y = fmaf(u.y, z.y, fmaf(u.w, z.w, su.y));
        sr.x = fmaf(r.x, x.x, fmaf(r.z, x.z, sr.x)), sr.y = fmaf(r.y, x.y, fmaf(r.w, x.w, sr.y));
        sw.x = fmaf(r.x, u.x, fmaf(r.z, u.z, sw.x)), sw.y = fmaf(r.y, u.y, fmaf(r.w, u.w, sw.y));
      }
      cp_wait<0>();
      __syncthreads();
      ws.load(w.dS + pt * NP, pr);  // on its way under the products
      ahead_of(h, p0);
      const float sx0 = -g.b[r0] * ex2(g.gh[r0]), sx1 = -g.b[r0 + 8] * ex2(g.gh[r0 + 8]);
      const float sk0 = decay_between(g, kC - 1, r0), sk1 = decay_between(g, kC - 1, r0 + 8);
      // a left operand of three planes with its rows scaled, as NL planes
      auto scaled = [&](uint32_t(&a)[NL][4], const uint32_t(&x)[3][4], float f0, float f1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo = 0.f, hi = 0.f;
#pragma unroll
          for (int l = 2; l >= 0; --l) {
            lo += __uint_as_float(x[l][e] << 16);
            hi += __uint_as_float(x[l][e] & 0xffff0000u);
          }
          const float f = e & 1 ? f1 : f0;
          uint32_t pp[NL];
          split2<NL>(lo * f, hi * f, pp);
#pragma unroll
          for (int l = 0; l < NL; ++l) a[l][e] = pp[l];
        }
      };
#pragma unroll 1  // (the code of one pass; four would miss the instruction cache)
      for (int kb = 0; kb < 4; ++kb) {
        uint32_t ya[NI][4], ra[3][4], xa[NL][4];
#pragma unroll
        for (int l = 0; l < NI; ++l) a_rows<kTP>(ya[l], yt + l * kC * kTP, strip * 16, kb * 16, lane);
#pragma unroll
        for (int l = 0; l < 3; ++l) a_cols<kTP>(ra[l], rt + l * kC * kTP, strip * 16, kb * 16, lane);
        scaled(xa, ra, sx0, sx1);
        if (kb == part) {  // dv = b dR: 16 of the value columns a warp
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = r0 + (e & 1) * 8, p = p0 + kb * 16 + (e >> 1) * 8 + c0;
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int l = 2; l >= 0; --l) {
              lo += __uint_as_float(ra[l][e] << 16);
              hi += __uint_as_float(ra[l][e] & 0xffff0000u);
            }
            if (i < rows && p < d.P)  // (rows from rv on are zeros)
              lm::st_two(dv + (tok + i) * ys + (int64_t)h * d.P + p,
                         make_float2(lo * g.b[i], hi * g.b[i]), p + 1 < d.P, d.wide);
          }
        }
        if (part <= strip) {
          auto ub = [&](int j, uint32_t(&x)[4]) {
            b_cols<kTP>(x, ut + j * kC * kTP, part * 16, kb * 16, lane);
          };
          mma_planes2<NI, 3, 3, 3, 3>(da[0], da[1], ya, wm[0], wm[1], ra, ub);
        }
#pragma unroll
        for (int np = 0; np < HT / 2; ++np) {
          auto sb = [&](int j, uint32_t(&x)[4]) {
            b_cols<LD>(x, st + j * kC * LD, part * WC + np * 16, kb * 16, lane);
          };
          mma_planes2<NI, 3, NL, NL, 3>(dqh[2 * np], dqh[2 * np + 1], ya, tk[2 * np], tk[2 * np + 1], xa,
                                        sb);
        }
      }
      __syncthreads();
      // dS over S0's place, and <dS, S0> of what is replaced
#pragma unroll
      for (int i = 0; i < ws.kN; ++i) {
        int r, cc;
        ws.at(i, &r, &cc);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int l = 2; l >= 0; --l) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(st + l * kC * LD + r * LD + cc);
          const uint32_t z = *reinterpret_cast<const uint32_t*>(st + l * kC * LD + (r + 8) * LD + cc);
          s.x += __uint_as_float(x << 16), s.y += __uint_as_float(x & 0xffff0000u);
          s.z += __uint_as_float(z << 16), s.w += __uint_as_float(z & 0xffff0000u);
        }
        const float4 v = ws.v[i];
        dot = fmaf(v.x, s.x, fmaf(v.y, s.y, fmaf(v.z, s.z, fmaf(v.w, s.w, dot))));
      }
      ws.template store<NL>(st);
      __syncthreads();
#pragma unroll 1  // (the code of one pass; four would miss the instruction cache)
      for (int kb = 0; kb < 4; ++kb) {
        uint32_t ua[3][4], xa[NL][4];
#pragma unroll
        for (int l = 0; l < 3; ++l) a_cols<kTP>(ua[l], ut + l * kC * kTP, strip * 16, kb * 16, lane);
        scaled(xa, ua, sk0, sk1);
#pragma unroll
        for (int np = 0; np < HT / 2; ++np)
          mma_planes<NL, NL, NL>(tk[2 * np], tk[2 * np + 1], xa, [&](int j, uint32_t(&x)[4]) {
            b_cols<LD>(x, st + j * kC * LD, part * WC + np * 16, kb * 16, lane);
          });
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) sm.dot[warp] = dot;
    auto halves = [&](float2 v, int which) {  // over the rows of a warp's loads
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
      static_assert(kGradThreads / 32 % 8 == 0, "every load of a thread has the same tokens");
      if (lane < 4)
        *reinterpret_cast<float2*>(&sm.part[warp >> 3][which][(warp & 7) * 8 + 2 * lane]) = v;
    };
    halves(su, 0);
    halves(sr, 1);
    halves(sw, 2);
    __syncthreads();  // the value tiles are read
    if constexpr (!SM::beside) {
      load_tile<T, NP, LD, kGradThreads>(qt, qg, d.qs, rv, d.N, d.vq);
      load_tile<T, NP, LD, kGradThreads>(kt, kg, d.ks, rv, d.N, d.vk);
      __syncthreads();
    }
    {  // the pairs of this warp: rows of its strip, 16 columns from part * 16 on
      float qk[2][4], kk[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) qk[t][e] = kk[t][e] = 0.f;
      if (part <= strip)
#pragma unroll 2
        for (int x = 0; x < NP / 16; ++x) {
          uint32_t qa[NI][4], ka[NI][4];
#pragma unroll
          for (int l = 0; l < NI; ++l) {
            a_rows<LD>(qa[l], qt + l * kC * LD, strip * 16, x * 16, lane);
            a_rows<LD>(ka[l], kt + l * kC * LD, strip * 16, x * 16, lane);
          }
          auto kb = [&](int j, uint32_t(&r)[4]) {
            b_rows<LD>(r, kt + j * kC * LD, part * 16, x * 16, lane);
          };
          mma_planes2<NI, NI, NI, NI, NI>(qk[0], qk[1], qa, kk[0], kk[1], ka, kb);
        }
      float rs[2] = {0.f, 0.f}, cs[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        cs[t][0] = cs[t][1] = 0.f;
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int i = r0 + e2 * 8, j = part * 16 + 8 * t + c0;
          float v1[2], v2[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int e = 2 * e2 + f;
            const float dec = j + f <= i ? decay_between(g, i, j + f) : 0.f;
            const float bd = j + f < i ? g.b[i] * dec : 0.f;
            v1[f] = d.scale * dec * da[t][e];
            v2[f] = -bd * wm[t][e];
            const float pair = v1[f] * qk[t][e] + v2[f] * kk[t][e];
            rs[e2] += pair;
            cs[t][f] += pair;
          }
          uint32_t x1[NL], x2[NL];
          split2<NL>(v1[0], v1[1], x1);
          split2<NL>(v2[0], v2[1], x2);
#pragma unroll
          for (int l = 0; l < NL; ++l) {
            *reinterpret_cast<uint32_t*>(p1 + l * kC * kTP + i * kTP + j) = x1[l];
            *reinterpret_cast<uint32_t*>(p2 + l * kC * kTP + i * kTP + j) = x2[l];
          }
        }
      }
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        rs[e2] += __shfl_xor_sync(0xffffffffu, rs[e2], 1);
        rs[e2] += __shfl_xor_sync(0xffffffffu, rs[e2], 2);
        if ((lane & 3) == 0) sm.row[part][r0 + e2 * 8] = rs[e2];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float v = cs[t][f];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane < 4) sm.col[strip][part * 16 + 8 * t + c0 + f] = v;
        }
    }
    {  // scale e^G q . (dY S0), and its part of dq
      const float f0 = d.scale * ex2(g.gh[r0]), f1 = d.scale * ex2(g.gh[r0 + 8]);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int t = 0; t < HT; ++t)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int i = r0 + e2 * 8, j = part * WC + 8 * t + c0;
          float qx = 0.f, qy = 0.f;
#pragma unroll
          for (int l = NI - 1; l >= 0; --l) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(qt + l * kC * LD + i * LD + j);
            qx += __uint_as_float(x << 16), qy += __uint_as_float(x & 0xffff0000u);
          }
          const float f = e2 ? f1 : f0, v0 = dqh[t][2 * e2] * f, v1 = dqh[t][2 * e2 + 1] * f;
          tq[t][2 * e2] += v0, tq[t][2 * e2 + 1] += v1;
          (e2 ? s1 : s0) += fmaf(v0, qx, v1 * qy);
        }
      s0 += __shfl_xor_sync(0xffffffffu, s0, 1), s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
      s0 += __shfl_xor_sync(0xffffffffu, s0, 2), s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
      if ((lane & 3) == 0) sm.qd[part][r0] = s0, sm.qd[part][r0 + 8] = s1;
    }
    __syncthreads();
#pragma unroll 1
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t a[NL][4], a2[NL][4];
      if (kb <= strip) {
#pragma unroll
        for (int l = 0; l < NL; ++l) {
          a_rows<kTP>(a[l], p1 + l * kC * kTP, strip * 16, kb * 16, lane);
          a_rows<kTP>(a2[l], p2 + l * kC * kTP, strip * 16, kb * 16, lane);
        }
#pragma unroll
        for (int np = 0; np < HT / 2; ++np) {
          auto kbl = [&](int j, uint32_t(&x)[4]) {
            b_cols<LD>(x, kt + j * kC * LD, part * WC + np * 16, kb * 16, lane);
          };
          mma_planes2<NL, max2(NL, NI), NL, max2(NL, NI), NI>(tq[2 * np], tq[2 * np + 1], a, tk[2 * np],
                                                              tk[2 * np + 1], a2, kbl);
        }
      }
      if (kb >= strip) {
#pragma unroll
        for (int l = 0; l < NL; ++l) {
          a_cols<kTP>(a[l], p1 + l * kC * kTP, strip * 16, kb * 16, lane);
          a_cols<kTP>(a2[l], p2 + l * kC * kTP, strip * 16, kb * 16, lane);
        }
#pragma unroll
        for (int np = 0; np < HT / 2; ++np) {
          mma_planes<NL, NI, max2(NL, NI)>(
              tk[2 * np], tk[2 * np + 1], a, [&](int j, uint32_t(&x)[4]) {
                b_cols<LD>(x, qt + j * kC * LD, part * WC + np * 16, kb * 16, lane);
              });
          mma_planes<NL, NI, max2(NL, NI)>(
              tk[2 * np], tk[2 * np + 1], a2, [&](int j, uint32_t(&x)[4]) {
                b_cols<LD>(x, kt + j * kC * LD, part * WC + np * 16, kb * 16, lane);
              });
        }
      }
    }
    if (warp == 0) {
      due = true;
      zd[0] = zt[0], zd[1] = zt[1];
#pragma unroll
      for (int x = 0; x < 2; ++x) bd[x] = g.b[2 * lane + x];
      ed = ex2(g.gh[kC - 1]);
    }
  }
  if (due) gates_of(h1 - 1);
  // padding rows are zeros: their keys, queries, corrections and gradients are
  const int64_t row = ((int64_t)b * d.T + t0 + r0) * d.G + grp, whole = (int64_t)d.B * d.T * d.G * d.N;
#pragma unroll
  for (int e2 = 0; e2 < 2; ++e2)
    if (r0 + 8 * e2 < rows) {
      const int64_t o = (row + (int64_t)8 * e2 * d.G) * d.N;
#pragma unroll
      for (int t = 0; t < HT; ++t) {
        const int j = part * WC + 8 * t + c0;
        const float2 vq = make_float2(tq[t][2 * e2], tq[t][2 * e2 + 1]);
        const float2 vk = make_float2(tk[t][2 * e2], tk[t][2 * e2 + 1]);
        if (j < d.N) {
          if (d.nb == 1) {
            lm::st_two(dq + o + j, vq, j + 1 < d.N, d.wide_k);
            lm::st_two(dk + o + j, vk, j + 1 < d.N, d.wide_k);
          } else {
            lm::st_two(w.dqp + hb * whole + o + j, vq, j + 1 < d.N, d.N % 2 == 0);
            lm::st_two(w.dkp + hb * whole + o + j, vk, j + 1 < d.N, d.N % 2 == 0);
          }
        }
      }
    }
}

// dq and dk as the sums of the head blocks' parts.
template <typename TO>
__global__ void __launch_bounds__(256)
    k_delta_sum(const float* __restrict__ qp, const float* __restrict__ kp, int nb, int64_t n,
                TO* __restrict__ dq, TO* __restrict__ dk) {
#pragma unroll 1
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float a = 0.f, b = 0.f;
    for (int l = 0; l < nb; ++l) a += qp[l * n + i], b += kp[l * n + i];
    dq[i] = from_f<TO>(a);
    dk[i] = from_f<TO>(b);
  }
}

// dA and ddt_bias of a head from the sums of its chunks, in a fixed order.
__global__ void __launch_bounds__(256)
    k_delta_params(const float* __restrict__ part, int B, int H, int nc, float* __restrict__ dA,
                   float* __restrict__ dbias) {
  __shared__ float s[2][8];
  const int h = blockIdx.x;
  float a = 0.f, b = 0.f;
  for (int n = 0; n < B; ++n) {
    const float2* p = reinterpret_cast<const float2*>(part) + ((int64_t)n * H + h) * nc;
#pragma unroll 4
    for (int i = threadIdx.x; i < nc; i += 256) {
      const float2 v = p[i];
      a += v.x, b += v.y;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if ((threadIdx.x & 31) == 0) s[0][threadIdx.x >> 5] = a, s[1][threadIdx.x >> 5] = b;
  __syncthreads();
  if (threadIdx.x == 0) {
    a = b = 0.f;
    for (int i = 0; i < 8; ++i) a += s[0][i], b += s[1][i];
    if (dA) dA[h] = a;
    if (dbias) dbias[h] = b;
  }
}

// ---------------------------------------------------------------------- host

// One part for each block of the heads of a group, so that the gradient's blocks fill
// the machine; each block sums its heads in registers.  Blocks, and forward and backward
// of 1 x 1024 and 1 x 256 tokens of 64 heads in 8 groups: gradient 152, outputs 608: 403 and
// 150 us; 304 and 1216: 409 and 135; 608 and 2432: 412 and 136.
constexpr int kGradBlocks = 2 * kRuleSms, kOutBlocks = 8 * kRuleSms;

// Segments of the chains: as many, up to 32 of at least 8 chunks, as make the modelled time
// shortest.  The model is of the forward's chain of bf16 inputs with 128 key columns, and every
// type, size and direction takes its choice, so that the states that the backward forms
// again are the forward's: a chunk of the chain takes 2.9 us with a block an SM and 5.1
// with two (which fit; 3.2 and 5.0 since a chunk's part of the state is summed apart); of the
// extra pass, which has the blocks of the moves as well and writes nothing on its way, 3.2
// with few blocks, 4.5 with up to two an SM and 3.8 for every two from there; a segment's
// join 3.8 us, more where the machine is full.  8192 tokens of 64 value rows, the three
// together: 8 heads 153 us, 16 163, 24 238; one segment takes 391, as of 48 heads, which are
// not cut.
void segments(DeltaDims* d) {
  const double heads = (double)d->B * d->H, vt = (d->Ps + kC - 1) / kC, mt = d->NP / kC;
  auto waves = [](double blocks) { return ceil(blocks / (2 * kRuleSms)); };
  auto chain = [&](double blocks) { return blocks <= kRuleSms ? 2.9 : 5.1 * waves(blocks); };
  auto ends = [&](double blocks) {
    return blocks <= 100 ? 3.2 : blocks <= 2 * kRuleSms ? 4.5 : 3.8 * waves(blocks);
  };
  d->W = 1, d->cs = d->nc;
  double best = d->nc * chain(heads * vt);
  for (int w = 2; w <= 32 && d->nc / w >= 8; w *= 2) {
    const int cs = (d->nc + w - 1) / w;
    const double join = heads * d->Ps / 16 / 100;
    const double t = cs * (ends(heads * (vt * (w - 1) + mt * (w - 2))) + chain(heads * vt * w)) +
                     3.8 * (w - 1) * (join < 1.0 ? 1.0 : join) + 8.0;
    if (t < 0.85 * best || (d->W > 1 && t < best)) best = t, d->W = w, d->cs = cs;
  }
}

int delta_dims(const ssd_delta_shape* s, DeltaDims* d) {
  if (!s || s->batch < 1 || s->seqlen < 1 || s->nheads < 1 || s->headdim < 1 || s->dstate < 1 ||
      s->ngroups < 1 || s->nheads % s->ngroups != 0)
    return SSD_ERR_INVALID_ARG;
  if ((s->in_dtype != SSD_F32 && s->in_dtype != SSD_BF16) ||
      (s->out_dtype != SSD_F32 && s->out_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  if (s->in_dtype == SSD_F32 && s->out_dtype == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  if (s->dstate > 128 || s->headdim > 256 || s->batch >= 65536 || s->nheads >= 65536 ||
      s->seqlen >= (1 << 30))
    return SSD_ERR_UNSUPPORTED;
  const int64_t gn = s->ngroups * s->dstate, hp = s->nheads * s->headdim;
  if ((s->q_row_stride && s->q_row_stride < gn) || (s->k_row_stride && s->k_row_stride < gn) ||
      (s->v_row_stride && s->v_row_stride < hp) || s->q_batch_stride < 0 ||
      s->k_batch_stride < 0 || s->v_batch_stride < 0)
    return SSD_ERR_INVALID_ARG;
  d->B = (int)s->batch, d->T = (int)s->seqlen, d->H = (int)s->nheads, d->G = (int)s->ngroups;
  d->P = (int)s->headdim, d->N = (int)s->dstate;
  d->rep = d->H / d->G;
  d->nc = (d->T + kC - 1) / kC;
  d->Ps = (d->P + 15) / 16 * 16;
  d->NP = d->N <= 64 ? 64 : 128;
  d->ip = s->in_dtype == SSD_BF16 ? 1 : 2;
  d->scale = s->scale;
  // a block for each (batch, head, chunk), or 64 value rows of a (batch, head)
  const int64_t bh = (int64_t)d->B * d->H;
  if (bh * d->nc >= 0x7fffffff || bh * 4 >= 0x7fffffff) return SSD_ERR_UNSUPPORTED;
  segments(d);
  const int64_t blocks = (int64_t)d->B * d->G * d->nc;
  int64_t nb = (kGradBlocks + blocks - 1) / blocks;
  if (s->out_dtype == SSD_F32) {
    // dk's accumulators take 12 accumulations a head and 8 for each 64 value rows, and each
    // truncates: 64 heads of bf16 inputs in one block were 2.7e-5 off, 8 are 4e-6, which
    // is the most here (a bf16 result's rounding is 2e-3)
    const int64_t most = 160 / (12 + 8 * ((d->Ps + kC - 1) / kC)), need = (d->rep + most - 1) / most;
    nb = nb > need ? nb : need;
  }
  d->nb = (int)(nb < d->rep ? nb : d->rep);
  const int64_t no = (kOutBlocks + blocks - 1) / blocks;
  d->no = (int)(no < d->rep ? no : d->rep);
  d->qs = s->q_row_stride ? s->q_row_stride : gn;
  d->ks = s->k_row_stride ? s->k_row_stride : gn;
  d->vs = s->v_row_stride ? s->v_row_stride : hp;
  d->qb = s->q_row_stride ? s->q_batch_stride : d->qs * d->T;
  d->kb = s->k_row_stride ? s->k_batch_stride : d->ks * d->T;
  d->vb = s->v_row_stride ? s->v_batch_stride : d->vs * d->T;
  return SSD_OK;
}

DeltaWs delta_ws(const DeltaDims& d, void* base, bool bwd) {
  DeltaWs w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    void* p = base ? static_cast<char*>(base) + at : nullptr;
    at += align_up(bytes, 256);
    return p;
  };
  const size_t n = (size_t)d.B * d.H * d.nc, tok = n * d.Ps * kC * 4, st = n * d.Ps * d.NP * 4;
  w.gates = static_cast<Gates*>(take(n * sizeof(Gates)));
  w.X = static_cast<bf16*>(take(n * 2 * kC * kTP * 2));
  const size_t image = (size_t)d.B * d.G * d.nc * d.ip * kC * (d.NP + 8) * 2;
  w.K = static_cast<bf16*>(take(image));
  w.U = static_cast<float*>(take(tok));
  w.S0 = static_cast<float*>(take(st));
  if (d.W > 1) {
    const size_t segs = (size_t)d.B * d.H * d.W * d.NP * 4;
    w.ends = static_cast<float*>(take(segs * d.Ps));
    w.front = static_cast<float*>(take(segs * d.Ps));
    w.move = static_cast<float*>(take(segs * d.NP));
  }
  if (bwd) {
    w.Q = static_cast<bf16*>(take(image));
    w.Zb = static_cast<float*>(take(tok));
    w.E = static_cast<float*>(take(tok));
    w.Zd = static_cast<float*>(take(tok));
    w.dR = static_cast<float*>(take(tok));
    w.dS = static_cast<float*>(take(st));
    w.part = static_cast<float*>(take(n * 8));
    if (d.nb > 1) {
      const size_t whole = (size_t)d.nb * d.B * d.T * d.G * d.N * 4;
      w.dqp = static_cast<float*>(take(whole));
      w.dkp = static_cast<float*>(take(whole));
    }
  }
  w.total = at;
  return w;
}

struct DeltaIn {
  const void *q, *k, *v, *dt;
  const float *dt_bias, *A;
  const void* beta;
  const float* init;
  const int32_t* lengths;
};
struct DeltaGrads {
  const void* dy;
  const float* dfinal;
  void *dq, *dk, *dv, *ddt, *dbeta;
  float *dA, *ddt_bias, *dinit;
};

template <typename K>
bool allow_smem(K kern, size_t bytes) {
  return bytes <= 48 * 1024 ||
         cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
             cudaSuccess;
}

// Launches kern and returns from the caller on an error.
#define DELTA_LAUNCH(name, kern, grid, threads, smem, ...)                       \
  do {                                                                           \
    if (!allow_smem(kern, smem)) return SSD_ERR_CUDA;                            \
    SSD_LAUNCH(name, s, kern<<<(unsigned)(grid), threads, smem, s>>>(__VA_ARGS__)); \
    if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;                  \
  } while (0)

template <typename T, int NP, bool BWD>
int delta_states(const DeltaDims& d, const DeltaIn& in, const void* dy, const DeltaWs& w,
                 float* final_states, cudaStream_t s) {
  const T *q = static_cast<const T*>(in.q), *k = static_cast<const T*>(in.k),
          *v = static_cast<const T*>(in.v);
  const int64_t n = (int64_t)d.B * d.H * d.nc, chains = (int64_t)d.B * d.H * ((d.Ps + kC - 1) / kC);
  const auto prep = k_delta_prep<T, NP, BWD>;
  DELTA_LAUNCH("k_delta_prep", prep, n, kPrepThreads, (PrepSmem<T, NP, BWD>::total), d, q, k,
               static_cast<const T*>(in.dt), in.dt_bias, in.A, static_cast<const T*>(in.beta),
               static_cast<const T*>(dy), in.lengths, w);
  if (d.W > 1) {
    const auto ends = k_delta_chain<T, NP, false, true>;
    DELTA_LAUNCH("k_delta_ends", ends, (int64_t)d.B * d.H * (d.W - 1) * ((d.Ps + kC - 1) / kC + NP / kC),
                 kChainThreads, (chain_smem<T, NP>()), d, v, in.init, in.lengths, w, nullptr,
                 device_status_ptr());
    DELTA_LAUNCH("k_delta_join", (k_delta_join<NP, false>), (int64_t)d.B * d.H * (d.Ps / 16), 4 * NP, 0, d, w);
  }
  const auto chain = k_delta_chain<T, NP, BWD, false>;
  DELTA_LAUNCH("k_delta_chain", chain, chains * d.W, kChainThreads, (chain_smem<T, NP>()), d, v, in.init,
               in.lengths, w, final_states, device_status_ptr());
  return SSD_OK;
}

template <typename T, typename TO, int NP>
int delta_forward(const DeltaDims& d, const DeltaIn& in, const DeltaWs& w, void* y,
                  float* final_states, cudaStream_t s) {
  const int st = delta_states<T, NP, false>(d, in, nullptr, w, final_states, s);
  if (st != SSD_OK) return st;
  const auto out = k_delta_out<T, TO, NP>;
  DELTA_LAUNCH("k_delta_out", out, (int64_t)d.B * d.G * d.no * d.nc, kOutThreads, (OutSmem<T, TO, NP>::total), d,
               static_cast<const T*>(in.q), static_cast<const T*>(in.k), in.lengths, w,
               static_cast<TO*>(y));
  return SSD_OK;
}

template <typename T, typename TO, int NP>
int delta_backward(const DeltaDims& d, const DeltaIn& in, const DeltaGrads& g, const DeltaWs& w,
                   cudaStream_t s) {
  const int st = delta_states<T, NP, true>(d, in, g.dy, w, nullptr, s);
  if (st != SSD_OK) return st;
  const T *q = static_cast<const T*>(in.q), *k = static_cast<const T*>(in.k),
          *dy = static_cast<const T*>(g.dy);
  const int64_t chains = (int64_t)d.B * d.H * ((d.Ps + kC - 1) / kC);
  if (d.W > 1) {
    const auto ends = k_delta_back<T, NP, true>;
    DELTA_LAUNCH("k_delta_back_ends", ends,
                 (int64_t)d.B * d.H * (d.W - 1) * ((d.Ps + kC - 1) / kC + NP / kC), kChainThreads,
                 (back_smem<T, NP>()), d, dy, g.dfinal, in.lengths, w, nullptr, device_status_ptr());
    DELTA_LAUNCH("k_delta_join", (k_delta_join<NP, true>), (int64_t)d.B * d.H * (d.Ps / 16), 4 * NP, 0, d,
                 w);
  }
  const auto back = k_delta_back<T, NP, false>;
  DELTA_LAUNCH("k_delta_back", back, chains * d.W, kChainThreads, (back_smem<T, NP>()), d, dy, g.dfinal,
               in.lengths, w, g.dinit, device_status_ptr());
  const auto grad = k_delta_grad<T, TO, NP>;
  TO *dq = static_cast<TO*>(g.dq), *dk = static_cast<TO*>(g.dk);
  DELTA_LAUNCH("k_delta_grad", grad, (int64_t)d.B * d.G * d.nb * d.nc, kGradThreads,
               (GradSmem<T, TO, NP>::total), d, q, k, static_cast<const T*>(in.dt), in.dt_bias, in.A, dy,
               in.lengths, w, dq, dk, static_cast<TO*>(g.dv), static_cast<TO*>(g.ddt),
               static_cast<TO*>(g.dbeta));
  if (d.nb > 1) {
    const int64_t m = (int64_t)d.B * d.T * d.G * d.N, blocks = (m + 255) / 256;
    DELTA_LAUNCH("k_delta_sum", k_delta_sum<TO>, blocks < kRuleSms * 8 ? blocks : kRuleSms * 8, 256, 0,
                 w.dqp, w.dkp, d.nb, m, dq, dk);
  }
  DELTA_LAUNCH("k_delta_params", k_delta_params, d.H, 256, 0, w.part, d.B, d.H, d.nc, g.dA,
               g.ddt_bias);
  return SSD_OK;
}

bool off(const void* p, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(esize - 1)) != 0;
}

// Whether rows of `cols` elements that start `step` elements apart at p, tokens row and
// batch rows batch elements apart, can be read 16 bytes at a time.
bool rows16(const void* p, int e, int64_t step, int64_t row, int64_t batch) {
  return !off(p, 16) && step * e % 16 == 0 && row * e % 16 == 0 && batch * e % 16 == 0;
}

int check_in(const ssd_delta_shape* shape, DeltaDims* d, const DeltaIn& in) {
  const int st = delta_dims(shape, d);
  if (st != SSD_OK) return st;
  const int e = shape->in_dtype == SSD_BF16 ? 2 : 4;
  if (!in.q || !in.k || !in.v || !in.dt || !in.A || !in.beta) return SSD_ERR_INVALID_ARG;
  if (off(in.q, e) || off(in.k, e) || off(in.v, e) || off(in.dt, e) || off(in.beta, e) ||
      off(in.dt_bias, 4) || off(in.A, 4) || off(in.init, 4) || off(in.lengths, 4))
    return SSD_ERR_INVALID_ARG;
  d->vq = rows16(in.q, e, d->N, d->qs, d->qb);
  d->vk = rows16(in.k, e, d->N, d->ks, d->kb);
  d->vv = rows16(in.v, e, d->P, d->vs, d->vb);
  return SSD_OK;
}

// Whether two tensors of states share memory: blocks of later segments write the last state
// while those of the first may still read the initial one.
bool overlap(const DeltaDims& d, const float* a, const float* b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && (x > y ? x - y : y - x) < (uintptr_t)d.B * d.H * d.P * d.N * sizeof(float);
}

int check_ws(const DeltaWs& w, const void* workspace, size_t bytes) {
  return !workspace || off(workspace, 16) || bytes < w.total ? SSD_ERR_WORKSPACE : SSD_OK;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

// The instance for the types and the key columns.
#define DELTA_PICK(call, ...)                                                             \
  (shape->in_dtype == SSD_F32                                                             \
       ? (d.NP == 64 ? call<float, float, 64>(__VA_ARGS__) : call<float, float, 128>(__VA_ARGS__)) \
   : shape->out_dtype == SSD_F32                                                          \
       ? (d.NP == 64 ? call<bf16, float, 64>(__VA_ARGS__) : call<bf16, float, 128>(__VA_ARGS__))   \
       : (d.NP == 64 ? call<bf16, bf16, 64>(__VA_ARGS__) : call<bf16, bf16, 128>(__VA_ARGS__)))

extern "C" {

size_t ssd_gated_delta_fwd_workspace_size(const ssd_delta_shape* shape) {
  DeltaDims d{};
  return delta_dims(shape, &d) == SSD_OK ? delta_ws(d, nullptr, false).total : 0;
}

size_t ssd_gated_delta_bwd_workspace_size(const ssd_delta_shape* shape) {
  DeltaDims d{};
  return delta_dims(shape, &d) == SSD_OK ? delta_ws(d, nullptr, true).total : 0;
}

int ssd_gated_delta_fwd(const ssd_delta_shape* shape, const void* q, const void* k, const void* v,
                        const void* dt, const float* dt_bias, const float* A, const void* beta,
                        const float* init_states, const int32_t* lengths, void* y,
                        float* final_states, void* workspace, size_t workspace_bytes,
                        void* stream) {
  DeltaDims d{};
  const DeltaIn in{q, k, v, dt, dt_bias, A, beta, init_states, lengths};
  int st = check_in(shape, &d, in);
  if (st != SSD_OK) return st;
  if (!y || off(y, shape->out_dtype == SSD_BF16 ? 2 : 4) || off(final_states, 4) ||
      overlap(d, init_states, final_states))
    return SSD_ERR_INVALID_ARG;
  d.wide = d.P % 2 == 0 && !off(y, shape->out_dtype == SSD_BF16 ? 4 : 8);
  const DeltaWs w = delta_ws(d, workspace, false);
  if ((st = check_ws(w, workspace, workspace_bytes)) != SSD_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return DELTA_PICK(delta_forward, d, in, w, y, final_states, s);
}

int ssd_gated_delta_bwd(const ssd_delta_shape* shape, const void* q, const void* k, const void* v,
                        const void* dt, const float* dt_bias, const float* A, const void* beta,
                        const float* init_states, const int32_t* lengths, const void* dy,
                        const float* dfinal_states, void* dq, void* dk, void* dv, void* ddt,
                        void* dbeta, float* dA, float* ddt_bias, float* dinit_states,
                        void* workspace, size_t workspace_bytes, void* stream) {
  DeltaDims d{};
  const DeltaIn in{q, k, v, dt, dt_bias, A, beta, init_states, lengths};
  int st = check_in(shape, &d, in);
  if (st != SSD_OK) return st;
  const int e = shape->in_dtype == SSD_BF16 ? 2 : 4, o = shape->out_dtype == SSD_BF16 ? 2 : 4;
  if (!dy || !dq || !dk || !dv || !ddt || !dbeta || off(dy, e) || off(dq, o) || off(dk, o) ||
      off(dv, o) || off(ddt, o) || off(dbeta, o) || off(dA, 4) || off(ddt_bias, 4) ||
      off(dfinal_states, 4) || off(dinit_states, 4) || overlap(d, dfinal_states, dinit_states))
    return SSD_ERR_INVALID_ARG;
  d.wide = d.P % 2 == 0 && !off(dv, 2 * o);
  d.wide_k = d.N % 2 == 0 && !off(dq, 2 * o) && !off(dk, 2 * o);
  d.vdy = rows16(dy, e, d.P, (int64_t)d.H * d.P, (int64_t)d.T * d.H * d.P);
  d.sms = sm_count();
  const DeltaWs w = delta_ws(d, workspace, true);
  if ((st = check_ws(w, workspace, workspace_bytes)) != SSD_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const DeltaGrads g{dy, dfinal_states, dq, dk, dv, ddt, dbeta, dA, ddt_bias, dinit_states};
  return DELTA_PICK(delta_backward, d, in, g, w, s);
}

}  // extern "C"
