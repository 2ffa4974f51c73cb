// Rotary angles of the calls that scale them: theta_i of a rotation's pairs, held as fractions of a turn, and
// the cosine and sine of a position's multiple of one, in fp32 or as pairs of fp32.
//
// A pair's theta / 2 pi goes to the kernels as a 64-bit binary fraction f; pos * f modulo 2^64 is the angle in
// turns, already reduced, by two integer products: no product in fp64, of which an SM does one warp
// instruction in 16 cycles.  f is off by theta / 2 pi times 3 2^-53 (the roundings of power, quotient and 2 pi) and by
// its own last half step, 2^-65; an angle by |pos| times that, below |pos| max(theta, 1) 2^-53 turns.
#pragma once

#include <math.h>

#include "common.cuh"

namespace csa2 {

constexpr int kMaxPairs = 256;

template <int kPairs>
struct Turns {
  uint64_t f[kPairs];
};

inline bool scaling_ok(const csa2_rope_scaling* s) {
  if (!s || s->kind == CSA2_SCALE_NONE) return true;
  if (s->kind != CSA2_SCALE_LINEAR && s->kind != CSA2_SCALE_YARN) return false;
  if (!(s->factor > 0.0f) || s->factor > 1.0e30f) return false;
  if (s->kind == CSA2_SCALE_LINEAR) return true;
  return s->original >= 1 && s->beta_slow > 0.0f && s->beta_fast > s->beta_slow && s->beta_fast <= 1.0e30f;
}

inline bool rotary_ok(const csa2_rotary* r, int64_t dim) {
  if (r->layout != CSA2_ROPE_INTERLEAVED && r->layout != CSA2_ROPE_HALVES) return false;
  if (r->n_rot < 2 || r->n_rot > 2 * kMaxPairs || r->n_rot % 2 != 0 || r->first < 0) return false;
  if ((int64_t)r->first + r->n_rot > dim) return false;
  if (!(r->base > 1.0f) || r->base > 1.0e30f) return false;
  return isfinite(r->magnitude) && scaling_ok(&r->scaling);
}

// theta of the pairs of a rotation of n channels
inline void make_thetas(double* t, int n, double base, const csa2_rope_scaling* s) {
  const int kind = s ? s->kind : CSA2_SCALE_NONE;
  double lo = 0.0, width = 1.0;
  if (kind == CSA2_SCALE_YARN) {
    const auto at = [&](double turns) {
      return n * log((double)s->original / (turns * 2.0 * 3.14159265358979323846)) / (2.0 * log(base));
    };
    lo = fmax(floor(at(s->beta_fast)), 0.0);
    width = fmax(fmin(ceil(at(s->beta_slow)), n - 1.0) - lo, 1e-3);
  }
  for (int i = 0; i < n / 2; ++i) {
    t[i] = pow(base, -2.0 * i / n);
    if (kind == CSA2_SCALE_LINEAR) t[i] /= (double)s->factor;
    if (kind == CSA2_SCALE_YARN) {
      const double ramp = fmin(fmax((i - lo) / width, 0.0), 1.0);
      t[i] = t[i] * (1.0 - ramp) + t[i] / (double)s->factor * ramp;
    }
  }
}
// theta / 2 pi of the pairs, as fractions of a turn
template <int kPairs>
inline void make_turns(Turns<kPairs>* t, int n, double base, const csa2_rope_scaling* s) {
  double theta[kPairs];
  make_thetas(theta, n, base, s);
  for (int i = 0; i < n / 2; ++i) {
    const double turns = theta[i] / 6.283185307179586476925286766559;
    t->f[i] = (uint64_t)rint((turns - floor(turns)) * 0x1p64);  // doubles of 2^53 and more are whole already
  }
}

// cosine and sine of pos times f, fp32: Taylor's series within an eighth of a turn, whose last terms are below 2^-28.
// The angle is rounded to 2^-24 of itself (at most pi / 4), each series to about two units of 2^-24.
__device__ __forceinline__ void turn_cos_sin(uint64_t f, int64_t pos, float& c, float& s) {
  const uint32_t phase = (uint32_t)(((uint64_t)pos * f) >> 32);
  const uint32_t quarter = (phase + (1u << 29)) >> 30;
  const float x = (float)(int32_t)(phase - (quarter << 30)) * (6.283185307179586f * 0x1p-32f), z = x * x;
  float sn = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f), cs = fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  sn = fmaf(x * z, fmaf(z, fmaf(z, sn, 1.0f / 120.0f), -1.0f / 6.0f), x);
  cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, cs, -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
  c = quarter & 1 ? sn : cs;
  s = quarter & 1 ? cs : sn;
  if ((quarter + 1) & 2) c = -c;
  if (quarter & 2) s = -s;
}

// ------------------------------------------------------------- pairs of fp32
// A value as the unevaluated sum hi + lo of two fp32, about 48 bits: sums by Knuth's TwoSum, products by an FMA's
// exact remainder (T. J. Dekker, "A floating-point technique for extending the available precision", Numer. Math. 18,
// 1971).  The _rn intrinsics keep the compiler from fusing what has to be rounded.
struct FF {
  float hi, lo;
};
__device__ __forceinline__ FF fast_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return FF{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ FF two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return FF{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ FF two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return FF{p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ FF mul(FF a, FF b) {
  const FF p = two_prod(a.hi, b.hi);
  return fast_sum(p.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, p.lo)));
}
__device__ __forceinline__ FF mul(FF a, float b) {
  const FF p = two_prod(a.hi, b);
  return FF{p.hi, __fmaf_rn(a.lo, b, p.lo)};
}
__device__ __forceinline__ FF add(FF a, FF b) {
  const FF s = two_sum(a.hi, b.hi);
  return fast_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ FF neg(FF a) { return FF{-a.hi, -a.lo}; }
// rounded once; a zero keeps its sign, and an infinity has no remainder
__device__ __forceinline__ float value(FF a) { return a.lo != 0.0f && isfinite(a.hi) ? __fadd_rn(a.hi, a.lo) : a.hi; }

// cosine and sine of a 64-bit fraction of a turn, to about 2^-38: Taylor's series within an eighth of a turn, the
// first terms in pairs of fp32, the rest (at most 2^-12 of the sum) in fp32
__device__ __forceinline__ void turn_cos_sin(uint64_t phase, FF& c, FF& s) {
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const int64_t r = (int64_t)(phase - ((uint64_t)quarter << 62));  // [-2^61, 2^61)
  const FF t = fast_sum((float)(int32_t)(r >> 40) * 0x1p-24f, (float)((uint32_t)(r >> 16) & 0xFFFFFFu) * 0x1p-48f);
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  constexpr FF two_pi{(float)kTwoPi, (float)(kTwoPi - (double)(float)kTwoPi)};
  const FF x = mul(t, two_pi), z = mul(x, x);
  constexpr auto inverse = [](double n) { return FF{(float)(1.0 / n), (float)(1.0 / n - (double)(float)(1.0 / n))}; };
  constexpr FF k6 = inverse(-6.0), k24 = inverse(24.0), k120 = inverse(120.0), k720 = inverse(-720.0);
  const float w = z.hi;
  float p = w * fmaf(w, fmaf(w, fmaf(w, 1.0f / 6227020800.0f, -1.0f / 39916800.0f), 1.0f / 362880.0f), -1.0f / 5040.0f);
  FF u = mul(add(k120, FF{p, 0.0f}), z);
  u = mul(add(k6, u), z);
  const FF sn = add(x, mul(x, u));
  p = w * fmaf(w, fmaf(w, 1.0f / 479001600.0f, -1.0f / 3628800.0f), 1.0f / 40320.0f);
  FF v = mul(add(k720, FF{p, 0.0f}), z);
  v = mul(add(k24, v), z);
  v = mul(add(FF{-0.5f, 0.0f}, v), z);
  const FF cs = add(FF{1.0f, 0.0f}, v);
  c = quarter & 1 ? sn : cs;
  s = quarter & 1 ? cs : sn;
  if (quarter == 1 || quarter == 2) c = neg(c);
  if (quarter >= 2) s = neg(s);
}
// (x, y) turned counter-clockwise; infinities, given or where the sum passes the largest fp32, have no remainders: in fp32
__device__ __forceinline__ void turn_pair(FF& x, FF& y, FF c, FF s) {
  FF nx = add(mul(x, c), neg(mul(y, s))), ny = add(mul(x, s), mul(y, c));
  if (!isfinite(x.hi) || !isfinite(y.hi) || !isfinite(nx.hi) || !isfinite(ny.hi)) {
    nx = FF{x.hi * c.hi - y.hi * s.hi, 0.0f};
    ny = FF{x.hi * s.hi + y.hi * c.hi, 0.0f};
  }
  x = nx;
  y = ny;
}

}  // namespace csa2
