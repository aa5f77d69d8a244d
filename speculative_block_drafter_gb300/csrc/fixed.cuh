// Softmax weights as whole numbers, for choices that have to fall on the exact
// side of a border: W = 2^40 e^((x - m) / T) rounded to the nearest integer, so
// that sums of up to 2^21 of them are exact in 64 bits whatever their order, a
// cumulative sum is the same however it is split, and u * sum compares without
// rounding. W is off by less than two (2^-39 of the largest weight): with f32
// weights, off by 2^-22, one choice in some hundred of a flat row of 150,000 would
// land beside its border.
//
// 2^y by a table of 2^(j / 64) and the Taylor series of 2^g, |g| <= 1/128, with
// y and g carried as unevaluated sums of two floats.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace dfl {

constexpr int FX_BITS = 40;

// 2^(j / 64) * 2^60.
static __device__ const unsigned long long kFxTable[64] = {
    0x1000000000000000ull, 0x102c9a3e778060eeull, 0x1059b0d31585743bull, 0x10874518759bc809ull,
    0x10b5586cf9890f63ull, 0x10e3ec32d3d1a202ull, 0x111301d0125b50a5ull, 0x11429aaea92ddfb3ull,
    0x1172b83c7d517addull, 0x11a35beb6fcb753dull, 0x11d4873168b9aa78ull, 0x12063b88628cd63cull,
    0x12387a6e75623867ull, 0x126b4565e27cdd25ull, 0x129e9df51fdee12cull, 0x12d285a6e4030b40ull,
    0x1306fe0a31b7152eull, 0x133c08b26416ff4dull, 0x1371a7373aa9caa7ull, 0x13a7db34e59ff6eaull,
    0x13dea64c12342236ull, 0x14160a21f72e29f8ull, 0x144e086061892d03ull, 0x1486a2b5c13cd014ull,
    0x14bfdad5362a271dull, 0x14f9b2769d2ca6adull, 0x15342b569d4f81dfull, 0x156f4736b527da67ull,
    0x15ab07dd48542959ull, 0x15e76f15ad21486full, 0x16247eb03a5584b2ull, 0x1662388255222491ull,
    0x16a09e667f3bcc91ull, 0x16dfb23c651a2ef2ull, 0x171f75e8ec5f73ddull, 0x175feb564267c8bfull,
    0x17a11473eb0186d8ull, 0x17e2f336cf4e6210ull, 0x182589994cce128bull, 0x1868d99b4492ec81ull,
    0x18ace5422aa0db5cull, 0x18f1ae991577362cull, 0x193737b0cdc5e4f4ull, 0x197d829fde4e4f8cull,
    0x19c49182a3f0901cull, 0x1a0c667b5de564b3ull, 0x1a5503b23e255c8bull, 0x1a9e6b5579fdbf44ull,
    0x1ae89f995ad3ad5full, 0x1b33a2b84f15faf7ull, 0x1b7f76f2fb5e46ebull, 0x1bcc1e904bc1d224ull,
    0x1c199bdd85529c22ull, 0x1c67f12e57d14b4aull, 0x1cb720dcef906915ull, 0x1d072d4a07897b8dull,
    0x1d5818dcfba48726ull, 0x1da9e603db328571ull, 0x1dfc97337b9b5eb9ull, 0x1e502ee78b3ff627ull,
    0x1ea4afa2a490d986ull, 0x1efa1bee615a2777ull, 0x1f50765b6e454067ull, 0x1fa7c1819e90d82full,
};

// log2(e) / T as a sum of two floats (kept finite for the smallest T > 0). In f32:
// an f64 division takes 16 cycles an instruction and warp on this GPU.
struct FxScale {
  float hi, lo;
};
__device__ __forceinline__ FxScale fx_scale(float T) {
  const float lh = 1.44269502f, ll = 1.92596303e-8f;             // log2(e) = lh + ll
  FxScale s;
  s.hi = lh / T;
  s.lo = 0.f;
  if (!(s.hi <= 1e30f)) s.hi = 1e30f;
  else if (s.hi > 1e-30f) s.lo = (fmaf(-s.hi, T, lh) + ll) / T;
  return s;
}

// The weight of a difference d + e <= 0 (an unevaluated sum, e at most a step of d); 0 for NaN. Without
// branches, so that several run side by side: below 2^-42 (and for NaN) y is -42, whose
// weight rounds to 0 whatever the low parts hold then (their part is below 2^-14).
// `tab`: kFxTable, in shared memory.
__device__ __forceinline__ unsigned long long fx_weight_diff(float d, float e, FxScale c, const unsigned long long *tab) {
  const float y = fmaxf(d * c.hi, -42.f);
  const float yl = fmaf(d, c.hi, -y) + fmaf(d, c.lo, e * c.hi);
  // (f32 numbers are rounded to whole ones by adding 1.5 * 2^23, except the one that
  // needs more bits: conversions to 64-bit integers take 16 cycles an instruction and
  // warp, those to 32 bits 2)
  const float big = 12582912.f, kb = fmaf(y, 64.f, big), k = kb - big;
  const float g = fmaf(k, -0.015625f, y);                        // exact
  const float ln2h = 0x1.62e4300000000p-1f, ln2l = -0x1.05c6100000000p-29f;
  const float x = g * ln2h;
  const float xl = fmaf(g, ln2h, -x) + fmaf(g, ln2l, yl * ln2h);
  // e^(x + xl) - 1 = x + (xl + x^2/2 + x^3/6 + x^4/24 + x xl)
  const float p = fmaf(x * x, fmaf(x, fmaf(x, 1.f / 24.f, 1.f / 6.f), 0.5f), fmaf(x, xl, xl));
  // x = fh 2^-29 + rest; the rest and p in steps of 2^-46 (|p| < 2^-15)
  const float hb = fmaf(x, 0x1p29f, big), rest = fmaf(hb - big, -0x1p-29f, x);
  const int fh = __float_as_int(hb) - 0x4B400000;
  const int fl = (int)((unsigned)__float2int_rn(p * 0x1p46f) + __float_as_uint(fmaf(rest, 0x1p46f, big)) - 0x4B400000u);
  const int ki = __float_as_int(kb) - 0x4B400000;
  const unsigned long long t = tab[ki & 63];
  const int th = (int)(t >> 30), tl = (int)((unsigned)t & 0x3fffffffu);
  const unsigned long long w =
      t + (unsigned long long)(((long long)fh * th << 1) + ((long long)fh * tl >> 29) + ((long long)fl * th >> 16));
  const int sh = 60 - FX_BITS - (ki >> 6);                       // 20 .. 62
  return (w + (1ull << (sh - 1))) >> sh;
}

// The weight of x against the largest value m (-inf: no value). NaN counts as
// -inf; against m = +inf, the infinite values share the weight.
__device__ __forceinline__ unsigned long long fx_weight(float x, float m, FxScale c, const unsigned long long *tab) {
  const float top = m > -INFINITY ? m : INFINITY;
  const float d = x == top ? 0.f : x - top, b = d - x;
  const float e = (x - (d - b)) + (-top - b);                    // d + e = x - m exactly
  return x > -INFINITY ? fx_weight_diff(d, e, c, tab) : 0ull;
}

// floor(f * n) for 0 <= f (NaN and negative: 0), saturated.
__device__ __forceinline__ unsigned long long fx_mul(float f, unsigned long long n) {
  if (!(f > 0.f)) return 0ull;
  if (f >= 16777216.f) return ~0ull;
  const int bits = __float_as_int(f), ex = bits >> 23;
  const unsigned long long man = ex ? (bits & 0x7fffff) | 0x800000 : (bits & 0x7fffff);
  const int sh = 150 - (ex ? ex : 1);                            // f = man * 2^-sh, sh >= 0
  const unsigned long long lo = man * n, hi = __umul64hi(man, n);
  if (sh == 0) return hi ? ~0ull : lo;
  if (sh < 64) return (hi >> sh) ? ~0ull : (hi << (64 - sh)) | (lo >> sh);
  return sh < 128 ? hi >> (sh - 64) : 0ull;
}
// The place of a uniform number (taken into [0, 1)) in a sum of weights: the
// choice is the first whose cumulative sum is above it.
__device__ __forceinline__ unsigned long long fx_target(float u, unsigned long long sum) {
  return fx_mul(fminf(u, 0.99999994f), sum);
}

// n / d of whole numbers below 2^62 (d > 0), rounded once (to within 2^-40 of a step).
__device__ __forceinline__ float fx_ratio(unsigned long long n, unsigned long long d) {
  const float nh = __ull2float_rn(n), nl = __ll2float_rn((long long)(n - __float2ull_rn(nh)));
  const float dh = __ull2float_rn(d), dl = __ll2float_rn((long long)(d - __float2ull_rn(dh)));
  const float h = nh / dh;
  return h + (fmaf(-h, dh, nh) + (nl - h * dl)) / dh;
}

}  // namespace dfl
