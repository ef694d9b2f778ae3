// Warp-level matrix pieces of the gated delta rule's chunk kernels: 16-bit products
// with fp32 accumulators (m16n8k16) whose operands are sums of 16-bit planes.
//
// An fp32 value v is the sum of the planes rn(v), rn(v - p0), rn(v - p0 - p1): 8
// significant bits each, so three planes hold v exactly up to 2^-25 of it.  A
// product of values with NA and NB planes takes the plane products i + j < max(NA,
// NB): a bf16 input (one plane, exact) times an fp32 value is three instructions and
// as good as an fp32 product, two fp32 values take six.  Chains of products stay in
// registers: an accumulator tile of 16 rows is, column block by column block, the
// left operand of the next product.
//
// Where rows can be scaled by a power of two first, two planes of fp16 do what three of
// bf16 do: with the row's largest value at the top of fp16's range, rn(v) and rn(v - p0)
// leave 2^-22 of v, or 2^-39 of the largest value where v is under 2^-17 of it (fp16's
// smallest step; with the largest at 1 that would begin 2^14 times higher), and a product
// of two such values takes three instructions (the lower planes' product is below).
//
// Operand tiles in shared memory are rows of 16-bit values with a pitch of an odd number of 16
// bytes, which ldmatrix reads without bank conflicts.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ssd {
namespace wm {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ uint32_t saddr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const bf16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr(p))
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const bf16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr(p))
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Lane addresses.  A (16 x 16) and B (16 x 16: two tiles of 8 columns) of a tile
// stored either way round; `ld` is the pitch in elements.
//   a_rows: stored [row][k]      a_cols: stored [k][row]
//   b_rows: stored [n][k]        b_cols: stored [k][n]
template <int LD>
__device__ __forceinline__ void a_rows(uint32_t (&r)[4], const bf16* t, int row, int k, int lane) {
  ldsm4(r, t + (row + (lane & 15)) * LD + k + (lane >> 4) * 8);
}
template <int LD>
__device__ __forceinline__ void a_cols(uint32_t (&r)[4], const bf16* t, int row, int k, int lane) {
  ldsm4t(r, t + (k + (lane & 7) + (lane >> 4) * 8) * LD + row + ((lane >> 3) & 1) * 8);
}
template <int LD>
__device__ __forceinline__ void b_rows(uint32_t (&r)[4], const bf16* t, int n, int k, int lane) {
  ldsm4(r, t + (n + (lane & 7) + (lane >> 4) * 8) * LD + k + ((lane >> 3) & 1) * 8);
}
template <int LD>
__device__ __forceinline__ void b_cols(uint32_t (&r)[4], const bf16* t, int n, int k, int lane) {
  ldsm4t(r, t + (k + (lane & 7) + ((lane >> 3) & 1) * 8) * LD + n + (lane >> 4) * 8);
}

// The planes of a pair of values, packed (first value in the low half).
template <int NPL>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&p)[NPL]) {
  float2 v = make_float2(a, b);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    p[i] = *reinterpret_cast<const uint32_t*>(&h);
    if (i + 1 < NPL) {  // what the plane leaves, exact in fp32
      const float2 f =
          make_float2(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xffff0000u));
      v = __ffma2_rn(f, make_float2(-1.f, -1.f), v);
    }
  }
}
// Left operand of column block kb of an accumulator strip c[tile][4], as planes.
template <int NPL, int NT>
__device__ __forceinline__ void a_from_acc(uint32_t (&a)[NPL][4], const float (&c)[NT][4], int kb) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t p[NPL];
    const float(&t)[4] = c[2 * kb + (q >> 1)];
    split2<NPL>(t[(q & 1) * 2], t[(q & 1) * 2 + 1], p);
#pragma unroll
    for (int i = 0; i < NPL; ++i) a[i][q] = p[i];
  }
}

// c0, c1 (two tiles of 8 columns) += A B over plane products i + j < M; B of plane j
// comes from load(j, regs).
// An accumulation truncates, which adds up where one accumulator takes many: of two fp32
// operands the lower products are summed apart (from zero, added by a rounded fp32 add),
// and the accumulator takes one product of the upper planes.  (Six into one: 3e-6 of an
// fp32 result; so: 6e-7.)
template <int NA, int NB, int M>
constexpr bool kApart = NA == 3 && NB == 3 && M == 3;
__device__ __forceinline__ void add4(float (&c)[4], const float (&t)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += t[e];
}
// The products with plane j of B, into the accumulator or what is summed apart.
template <int NA, int M, bool APART>
__device__ __forceinline__ void plane_products(float (&c0)[4], float (&c1)[4], float (&t0)[4],
                                               float (&t1)[4], const uint32_t (&a)[NA][4],
                                               const uint32_t (&b)[4], int j) {
#pragma unroll
  for (int n = 0; n < NA; ++n) {
    const int i = APART ? NA - 1 - n : n;  // apart: the upper planes' product last
    if (i + j < M) {
      if constexpr (APART) {
        if (i + j > 0) {
          mma16816(t0, a[i], b[0], b[1]);
          mma16816(t1, a[i], b[2], b[3]);
          continue;
        }
        add4(c0, t0);
        add4(c1, t1);
      }
      mma16816(c0, a[i], b[0], b[1]);
      mma16816(c1, a[i], b[2], b[3]);
    }
  }
}
template <int NA, int NB, int M, typename Load>
__device__ __forceinline__ void mma_planes(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4],
                                           Load&& load) {
  float t0[4] = {}, t1[4] = {};
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int j = kApart<NA, NB, M> ? NB - 1 - n : n;
    uint32_t b[4];
    load(j, b);
    plane_products<NA, M, kApart<NA, NB, M>>(c0, c1, t0, t1, a, b, j);
  }
}

// ----------------------------------------------------------- fp16, rows scaled

// Power of two that brings the largest value m of a row to [2^14, 2^15), the top of fp16's
// range, and its inverse (m under 2^-112: 2^126).  An infinite value leaves nothing of the
// others of its row: the inverse is NaN, and so are the row's products.
struct Scale {
  float s, inv;
};
__device__ __forceinline__ Scale scale_of(float m) {
  const uint32_t e = max(__float_as_uint(m) >> 23, 15u);
  Scale r;
  r.s = __uint_as_float((268 - e) << 23);
  r.inv = __uint_as_float(e < 255 ? (e - 14) << 23 : 0x7fffffffu);
  return r;
}
// The planes of a pair of values times f.
__device__ __forceinline__ void split2h(float a, float b, float f, uint32_t (&p)[2]) {
  const float2 v = __fmul2_rn(make_float2(a, b), make_float2(f, f));
  const __half2 h = __float22half2_rn(v);
  const __half2 l = __float22half2_rn(__ffma2_rn(__half22float2(h), make_float2(-1.f, -1.f), v));
  p[0] = *reinterpret_cast<const uint32_t*>(&h);
  p[1] = *reinterpret_cast<const uint32_t*>(&l);
}
// Left operand of column block kb of an accumulator strip whose rows (lane / 4, + 8)
// are scaled by f0 and f1.
template <int NT>
__device__ __forceinline__ void a_from_acc_h(uint32_t (&a)[2][4], const float (&c)[NT][4], int kb,
                                             float f0, float f1) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t p[2];
    const float(&t)[4] = c[2 * kb + (q >> 1)];
    split2h(t[(q & 1) * 2], t[(q & 1) * 2 + 1], q & 1 ? f1 : f0, p);
    a[0][q] = p[0], a[1][q] = p[1];
  }
}
// Largest magnitudes of the strip's rows lane / 4 and lane / 4 + 8.
template <int NT>
__device__ __forceinline__ void row_max(const float (&c)[NT][4], float& m0, float& m1) {
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    a[t & 1] = fmaxf(fmaxf(a[t & 1], fabsf(c[t][0])), fabsf(c[t][1]));
    a[2 + (t & 1)] = fmaxf(fmaxf(a[2 + (t & 1)], fabsf(c[t][2])), fabsf(c[t][3]));
  }
  m0 = fmaxf(a[0], a[1]), m1 = fmaxf(a[2], a[3]);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
}
// c0, c1 += A B over planes: A of two, B of NB.
template <int NB, typename Load>
__device__ __forceinline__ void mma_planes_h(float (&c0)[4], float (&c1)[4],
                                             const uint32_t (&a)[2][4], Load&& load) {
#pragma unroll
  for (int j = NB - 1; j >= 0; --j) {
    uint32_t b[4];
    load(j, b);
#pragma unroll
    for (int i = 1; i >= 0; --i)
      if (i + j < 2) {
        mma16816h(c0, a[i], b[0], b[1]);
        mma16816h(c1, a[i], b[2], b[3]);
      }
  }
}

// The same right operand in two products: c0, c1 += A B over plane products i + j < M,
// e0, e1 += F B over i + j < ME.
template <int NA, int M, int NF, int ME, int NB, typename Load>
__device__ __forceinline__ void mma_planes2(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4],
                                            float (&e0)[4], float (&e1)[4], const uint32_t (&f)[NF][4],
                                            Load&& load) {
  constexpr bool APART = kApart<NA, NB, M> && kApart<NF, NB, ME>;  // both of fp32 operands
  float t0[4] = {}, t1[4] = {}, u0[4] = {}, u1[4] = {};
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int j = APART ? NB - 1 - n : n;
    uint32_t b[4];
    load(j, b);
    plane_products<NA, M, APART>(c0, c1, t0, t1, a, b, j);
    plane_products<NF, ME, APART>(e0, e1, u0, u1, f, b, j);
  }
}

constexpr int max2(int a, int b) { return a > b ? a : b; }

}  // namespace wm
}  // namespace ssd
