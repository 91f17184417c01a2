// The softmax half of attention tiles whose products run on tcgen05: of the
// prompt kernel and of the paged kernel for many new tokens.
//
// A warpgroup (four warps) owns a tile of 128 query rows, one row per thread.
// Its logits S (128 x 128 keys, fp32) lie in TMEM; the weights P go back as
// 16-bit values over S's first 64 columns, where the second product reads
// them as its A operand, and the output accumulator O (128 x D, fp32) stays in
// TMEM until the end.
//
// The exponent's reference is the running maximum, but it moves (and O and the
// running sum are rescaled) only when the maximum has grown by more than
// 2^kSlack since: weights then stay below 2^kSlack, which both 16-bit types and
// the fp32 sums hold without loss, and after the first tiles O is hardly ever
// read back.
//
// A tile's chain (logits, softmax, weighted sum, next logits) is what bounds
// both kernels, so the weights are handed over in two halves: the second
// product starts on the first 64 keys while the others' weights are computed.
//
// 128 x 128 exponentials cost the special-function units as many cycles as
// the tile's two products cost the tensor cores, so in the prompt kernel some of
// them run on the FMA pipe instead (ex2_poly2).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_sm100.cuh"

namespace tq {
namespace flash {

constexpr float kSlack = 8.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}

// 2^x of two values on the FMA pipe: x = n + f with n the nearest integer
// (round to nearest by adding 1.5 2^23) and |f| <= 1/2, 2^f by a polynomial
// times 2^n made from n's bits.  Below -127 the result is 0 exactly (2^-127's
// exponent field is 0) and a NaN stays one.  Coefficients: minimax fit of the relative error
// over |f| <= 1/2, largest error 2^-13.2 (degree 3, for bf16 weights, rounded
// at 2^-9) and 2^-18.4 (degree 4, for fp16 weights, rounded at 2^-12).
template <bool BF16>
__device__ __forceinline__ float2 ex2_poly2(float2 x) {
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.x));  // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.y));
  const float2 magic = make_float2(12582912.f, 12582912.f);
  const float2 t = add2(x, magic);
  const float2 n = add2(t, make_float2(-12582912.f, -12582912.f));
  const float2 f = fma2(n, make_float2(-1.f, -1.f), x);
  float2 p;
  if constexpr (BF16) {
    p = fma2(f, make_float2(0.05500893294811249f, 0.05500893294811249f), make_float2(0.2422109693288803f, 0.2422109693288803f));
    p = fma2(f, p, make_float2(0.6932829022407532f, 0.6932829022407532f));
  } else {
    p = fma2(f, make_float2(0.009582852944731712f, 0.009582852944731712f), make_float2(0.055906426161527634f, 0.055906426161527634f));
    p = fma2(f, p, make_float2(0.24024099111557007f, 0.24024099111557007f));
    p = fma2(f, p, make_float2(0.6931241750717163f, 0.6931241750717163f));
  }
  p = fma2(f, p, make_float2(1.f, 1.f));
  return mul2(p, make_float2(__uint_as_float(0x3F800000u + (__float_as_uint(t.x) << 23)),
                             __uint_as_float(0x3F800000u + (__float_as_uint(t.y) << 23))));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float2 v) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}

// One row's running softmax state, in base 2: the exponent's reference and the
// sum of the weights.  The reference has two parts, a logit and (of the paged
// cache, 0 otherwise) the exponent of a value norm: what a value is multiplied by,
// weight times norm, is what stays below 2^kSlack.  They are kept apart because
// beside a large logit the exponent would be lost in a sum, from the weights but
// not from the values.  The sum, relative to both, may be as large as 2^80 a key
// and as small as 2^-100: see move_reference.
struct Row {
  float ref = -INFINITY, norm = 0.f, sum = 0.f;
  __device__ float exponent() const { return ref + norm; }  // of sum and O
};

// Exponent e of a value norm v below 2^e (v >= 0), no less than -80 (a weight is at
// most 2^8 over its key's norm, and the sum of 2^29 of them has to fit fp32)
__device__ __forceinline__ float norm_exponent(float v) {
  return fmaxf(__uint_as_float((__float_as_uint(v) >> 23) + 0x4B000000u) - (8388608.f + 126.f), -80.f);
}

// O *= f, one row per thread (whole warps)
template <int D>
__device__ __forceinline__ void scale_rows(uint32_t o, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t v[32];
    sm100::tmem_ld32(o + c, v);
    sm100::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
    sm100::tmem_st32(o + c, v);
  }
  sm100::tmem_wait_st();
}

// From logits this large (base 2) on the fused a * mult - reference differs from
// the rounded product that the reference is by more than an fp16 weight near 1 is
// rounded by (2^-12), and from 2^28 on the weights would leave fp32.  Such a row's
// products are rounded first, so that its highest logit's weight is 1.  In the paged
// cache's kernel, where they cost a warp two more passes, from 2^16 on alone.
constexpr float kLargeRow = 4096.f, kLargeLogit = 65536.f;

// Moves a row's reference up to a tile's highest logit (base 2) and the exponent
// of the values there, where the two together have grown by more than the slack;
// sum and O follow (the sum by a root of the factor twice: a factor of 2^-126 or
// less is 0, and the sum may be 2^180 above what it is then added to).  first: O is
// not there yet.  Whether a row moves, and by how much, is its own affair: moving
// all rows of a warp with the first that has to would put its neighbours, rows
// that it does not see among them, into a row's roundings.  Returns whether the
// row has large logits; SMALL: whether any of the warp has, and nothing is moved.
template <int D, bool SMALL>
__device__ __forceinline__ bool move_reference(uint32_t o, bool first, float most, float norm, Row &row) {
  const float up = (most - row.ref) + (norm - row.norm);  // infinite for the first visible keys, a NaN for none so far
  const float top = fmaxf(most, row.ref);
  const bool large = fabsf(top) > (SMALL ? kLargeLogit : kLargeRow) && top > -INFINITY;
  if (!__any_sync(0xffffffffu, up > kSlack || large)) return false;
  if (SMALL && __any_sync(0xffffffffu, large)) return true;
  float f = 1.f;
  if (up > kSlack) {
    f = ex2(-0.5f * up);
    row.ref = most;
    row.norm = norm;
  }
  row.sum = f * row.sum * f;
  if (!first && __any_sync(0xffffffffu, f != 1.f)) scale_rows<D>(o, f * f);
  return large;
}

// Weights are in TMEM: the product that reads them may start
__device__ __forceinline__ void hand_over(uint64_t *bar) {
  sm100::tmem_wait_st();
  sm100::tc_fence_before();
  sm100::mbar_arrive(bar);
}

// One tile of 128 keys: S at `s` -> P over it, handed over by halves (64 keys
// each) on two barriers.  mult >= 0 turns logits into base-2 exponents.  MASK:
// the row sees the tile's first `see` keys alone.  PAIRS of eight pairs of
// exponentials run on the FMA pipe (prompts of 8192 tokens, d = 128: with 2 968
// us, with 3 or 4 992).  The row's 128 logits stay in registers: reading S
// twice, 32 columns at a time, took 1040 us instead of 968.
template <int D, bool BF16, bool MASK, int PAIRS>
__device__ __forceinline__ void softmax_tile(uint32_t s, uint32_t o, bool first, float mult, int see, Row &row,
                                             uint64_t *half, uint64_t *full) {
  float x[128];
  uint32_t(*v)[32] = reinterpret_cast<uint32_t(*)[32]>(x);
#pragma unroll
  for (int c = 0; c < 4; ++c) sm100::tmem_ld32(s + 32 * c, v[c]);
  sm100::tmem_wait_ld();
  if constexpr (MASK) {
#pragma unroll
    for (int i = 0; i < 128; ++i) x[i] = i < see ? x[i] : -INFINITY;
  }
  float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 4; i < 124; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], fmaxf(x[i + k], x[i + 4 + k]));
#pragma unroll
  for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], x[124 + k]);
  const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * mult;
  const bool large = move_reference<D, false>(o, first, most, 0.f, row);
  const float base = row.ref == -INFINITY ? 0.f : -row.ref;
  if (large) {
#pragma unroll
    for (int i = 0; i < 128; ++i) x[i] *= mult;
    mult = 1.f;
  }
  __syncwarp();
  const float2 m2 = make_float2(mult, mult), b2 = make_float2(base, base);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int k = 64 * h + 2 * i;
      float2 e = fma2(make_float2(x[k], x[k + 1]), m2, b2);
      if (i % 8 >= 8 - PAIRS)
        e = ex2_poly2<BF16>(e);
      else
        e = make_float2(ex2(e.x), ex2(e.y));
      sum[i & 1] = add2(sum[i & 1], e);
      w[i] = pack16<BF16>(e);
    }
    sm100::tmem_st32(s + 32 * h, w);
    hand_over(h == 0 ? half : full);
  }
  row.sum += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The same with fp16 weights for the paged cache.  S is read twice, for the
// maximum and for the weights, 32 columns at a time, each read issued before the
// columns in hand are worked on: the warps that expand operands leave no
// registers for a row of 128 logits.  (P's columns reach no further than S's
// that are read already.)  The tile's values come scaled down by 2^scale, which
// the weights take back: the reference is of weight times 2^scale, so that P
// times the operand, in units of the reference, is what O adds up, whatever the
// other tiles' scales.  (All exponentials on the special-function unit: the
// expansion leaves no issue slots to spare; 512 new tokens on 16384 keys, us,
// with 0 of eight pairs on the FMA pipe 271, with 1 275, 2 281, 3 284.)
//
// keys: a factor of each key's logit in shared memory, below 0 where there is no
// such key; under MASK these are left out.  EACH: the factors are not all one, and
// each key's values are scaled down by a factor of their own, kFactors behind it
// (its exponent kFactors further on), in place of 2^scale.  A warp with large
// logits does nothing and returns false: softmax_tile_own then takes the tile.
constexpr int kFactors = 8 * 128;
template <bool MASK, bool EACH>
__device__ __forceinline__ void hide(float (&x)[32], int col, int see, const float *keys) {
  if constexpr (EACH) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float4 k = *reinterpret_cast<const float4 *>(keys + col + i);
      const float2 a = mul2(make_float2(x[i], x[i + 1]), make_float2(k.x, k.y));
      const float2 b = mul2(make_float2(x[i + 2], x[i + 3]), make_float2(k.z, k.w));
      x[i] = MASK && (k.x < 0.f || col + i >= see) ? -INFINITY : a.x;
      x[i + 1] = MASK && (k.y < 0.f || col + i + 1 >= see) ? -INFINITY : a.y;
      x[i + 2] = MASK && (k.z < 0.f || col + i + 2 >= see) ? -INFINITY : b.x;
      x[i + 3] = MASK && (k.w < 0.f || col + i + 3 >= see) ? -INFINITY : b.y;
    }
  } else if constexpr (MASK) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float4 k = *reinterpret_cast<const float4 *>(keys + col + i);
      x[i] = k.x < 0.f || col + i >= see ? -INFINITY : x[i];
      x[i + 1] = k.y < 0.f || col + i + 1 >= see ? -INFINITY : x[i + 1];
      x[i + 2] = k.z < 0.f || col + i + 2 >= see ? -INFINITY : x[i + 2];
      x[i + 3] = k.w < 0.f || col + i + 3 >= see ? -INFINITY : x[i + 3];
    }
  }
}
template <int D, bool MASK, bool EACH>
__device__ __forceinline__ bool softmax_tile_twice(uint32_t s, uint32_t o, bool first, float mult, int see, Row &row,
                                                   const float *keys, float scale, uint64_t *half, uint64_t *full) {
  uint32_t buf[2][32];
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  sm100::tmem_ld32(s, buf[0]);
#pragma unroll 2
  for (int c = 0; c < 4; ++c) {
    sm100::tmem_wait_ld();
    sm100::tmem_ld32(s + 32 * ((c + 1) & 3), buf[(c + 1) & 1]);
    float(&x)[32] = reinterpret_cast<float(&)[32]>(buf[c & 1]);
    hide<MASK, EACH>(x, 32 * c, see, keys);
    if constexpr (EACH) {
      const float4 *exps = reinterpret_cast<const float4 *>(keys + 2 * kFactors + 32 * c);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 n = exps[i / 4];
        const float2 a = fma2(make_float2(x[i], x[i + 1]), make_float2(mult, mult), make_float2(n.x, n.y));
        const float2 b = fma2(make_float2(x[i + 2], x[i + 3]), make_float2(mult, mult), make_float2(n.z, n.w));
        x[i] = a.x, x[i + 1] = a.y, x[i + 2] = b.x, x[i + 3] = b.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 32; i += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], fmaxf(x[i + k], x[i + 4 + k]));
  }
  const float highest = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * (EACH ? 1.f : mult);
  sm100::tmem_wait_ld();
  if (EACH) scale = 0.f;  // (in `highest` already)
  if (move_reference<D, true>(o, first, highest, scale, row)) return false;
  const float base = scale - row.norm - (row.ref == -INFINITY ? 0.f : row.ref);
  const float2 m2 = make_float2(mult, mult), b2 = make_float2(base, base);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 2
  for (int c = 0; c < 4; ++c) {
    sm100::tmem_wait_ld();
    if (c < 3) sm100::tmem_ld32(s + 32 * (c + 1), buf[(c + 1) & 1]);
    float(&x)[32] = reinterpret_cast<float(&)[32]>(buf[c & 1]);
    hide<MASK, EACH>(x, 32 * c, see, keys);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float2 e = fma2(make_float2(x[2 * i], x[2 * i + 1]), m2, b2);
      e = make_float2(ex2(e.x), ex2(e.y));
      sum[i & 1] = add2(sum[i & 1], e);
      if constexpr (EACH) e = mul2(e, *reinterpret_cast<const float2 *>(keys + kFactors + 32 * c + 2 * i));
      w[i] = pack16<false>(e);
    }
    sm100::tmem_st16(s + 16 * c, w);
    if (c & 1) hand_over(c == 1 ? half : full);
  }
  const float total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
  row.sum += EACH ? total : total * ex2(-scale);
  return true;
}

// The same tile with a factor of each key's logit, `keys`, and with values scaled
// down by a factor of each key's own, kFactors behind it.  Products are rounded
// before the reference is subtracted.  Three passes over S: the highest logit,
// the largest weight times norm relative to it, the weights.  A function of its
// own for tiles that are rare (norms far apart, large logits).
__device__ __forceinline__ void own_logits(uint32_t s, int c, float mult, int see, const float *keys, float (&x)[32]) {
  sm100::tmem_ld32(s + 32 * c, reinterpret_cast<uint32_t(&)[32]>(x));
  sm100::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float k = keys[32 * c + i];
    x[i] = k < 0.f || 32 * c + i >= see ? -INFINITY : __fmul_rn(x[i] * k, mult);
  }
}
template <int D>
__device__ __noinline__ Row softmax_tile_own(uint32_t s, uint32_t o, bool first, float mult, int see, Row row,
                                             const float *keys, uint64_t *half, uint64_t *full) {
  const float *values = keys + kFactors;
  float x[32], highest = -INFINITY, norm = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    own_logits(s, c, mult, see, keys, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) highest = fmaxf(highest, x[i]);
  }
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    own_logits(s, c, mult, see, keys, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) norm = fmaxf(norm, x[i] - highest + norm_exponent(values[32 * c + i]));
  }
  move_reference<D, false>(o, first, highest, norm, row);
  const float ref = row.ref == -INFINITY ? 0.f : row.ref;
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    own_logits(s, c, mult, see, keys, x);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 e = make_float2(ex2(x[2 * i] - ref - row.norm), ex2(x[2 * i + 1] - ref - row.norm));
      sum += e.x + e.y;
      w[i] = pack16<false>(mul2(e, *reinterpret_cast<const float2 *>(values + 32 * c + 2 * i)));
    }
    sm100::tmem_st16(s + 16 * c, w);
    if (c & 1) hand_over(c == 1 ? half : full);
  }
  row.sum += sum;
  return row;
}

}  // namespace flash
}  // namespace tq
