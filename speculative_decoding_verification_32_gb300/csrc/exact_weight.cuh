// exact_weight.cuh -- softmax weights exp((l - M) / T) of a row in two fp32 words.
//
// Where a sum of weights decides something (which token a uniform falls on, which
// logits top-p keeps), fp32 weights leave the answer open in one row of some
// dozens or hundreds.  These hold a weight to 2^-36 of itself (at most 2^-36.7 off in 10^7
// weights of random logits and temperatures, as far as 2^-36; below that the lower word
// runs into fp32's subnormal numbers, and weights of 2^-126 and less are 0), and a
// weight of 1 is 1.  fp64's own exp runs at a sixty-fourth of fp32's rate here.
//
// The method is table-driven reduction (P. T. P. Tang, "Table-driven implementation
// of the exponential function in IEEE floating-point arithmetic", 1989) with sums
// and products carried in two words by their exact remainders (T. J. Dekker, 1971;
// D. E. Knuth's sum of two numbers):  with y = (l - M) log2(e) / T
//   2^y = 2^n 2^(j/32) e^x,  y = n + j/32 + r,  |r| <= 1/64,  x = r ln 2,
// 2^(j/32) from a table of 32 two-word numbers and e^x - 1 = x + x^2/2 + .. + x^5/120
// (the next term is below 2^-48; x^2 is rounded at 2^-38).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sv {

// 2^(j/32): nearest fp32 number, and the nearest to what is left
__device__ const float2 kPower32[32] = {
    {0x1p0f, 0x0p0f}, {0x1.059b0ep0f, -0x1.9d4f52p-25f}, {0x1.0b5586p0f, 0x1.9f3122p-25f}, {0x1.11301ep0f, -0x1.fdb496p-25f},
    {0x1.172b84p0f, -0x1.c15742p-27f}, {0x1.1d4874p0f, -0x1.d2e8cap-25f}, {0x1.2387a6p0f, 0x1.ceac48p-25f}, {0x1.29e9ep0f, -0x1.5c0424p-25f},
    {0x1.306fep0f, 0x1.4636e2p-25f}, {0x1.371a74p0f, -0x1.18aac6p-25f}, {0x1.3dea64p0f, 0x1.824684p-25f}, {0x1.44e086p0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep0f, -0x1.593abcp-25f}, {0x1.5342b6p0f, -0x1.2c561p-25f}, {0x1.5ab07ep0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp0f, -0x1.f8b55p-25f},
    {0x1.6a09e6p0f, 0x1.9fcef4p-26f}, {0x1.71f75ep0f, 0x1.1d8beep-25f}, {0x1.7a1148p0f, -0x1.829fdp-25f}, {0x1.82589ap0f, -0x1.accc7cp-26f},
    {0x1.8ace54p0f, 0x1.15506ep-27f}, {0x1.93737cp0f, -0x1.e64744p-25f}, {0x1.9c4918p0f, 0x1.51f848p-27f}, {0x1.a5503cp0f, -0x1.b83b54p-25f},
    {0x1.ae89fap0f, -0x1.a94b14p-26f}, {0x1.b7f77p0f, -0x1.a09438p-25f}, {0x1.c199bep0f, -0x1.3d56b2p-27f}, {0x1.cb720ep0f, -0x1.8837ccp-27f},
    {0x1.d5818ep0f, -0x1.822dbcp-27f}, {0x1.dfc974p0f, -0x1.908c94p-25f}, {0x1.ea4afap0f, 0x1.52486cp-27f}, {0x1.f50766p0f, -0x1.246ebp-26f}};

// Two numbers side by side, where an instruction takes two (plain ones run at half the
// rate of these).
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 minus2(float2 a, float2 b) { return ffma2(b, both(-1.f), a); }
// a + b, and what the sum lost
__device__ __forceinline__ float two_sum(float a, float b, float &lost) {
  const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
  lost = __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v));
  return s;
}
__device__ __forceinline__ float2 two_sum(float2 a, float2 b, float2 &lost) {
  const float2 s = fadd2(a, b), v = minus2(s, a);
  lost = fadd2(minus2(a, minus2(s, v)), minus2(b, v));
  return s;
}
// ... where a is the larger one
__device__ __forceinline__ float fast_two_sum(float a, float b, float &lost) {
  const float s = __fadd_rn(a, b);
  lost = __fadd_rn(__fsub_rn(a, s), b);
  return s;
}

// A sum in two words, hi the nearest fp32 number to it (fp64 adds run at a sixty-fourth
// of fp32's rate).  Good to 2^-46 of itself.
struct alignas(8) Words {  // (sent to other CTAs in one piece)
  float hi, lo;
};
__device__ __forceinline__ Words add_words(Words a, Words b) {
  Words r;
  float e;
  const float s = two_sum(a.hi, b.hi, e);
  r.hi = fast_two_sum(s, __fadd_rn(e, __fadd_rn(a.lo, b.lo)), r.lo);
  return r;
}
__device__ __forceinline__ Words times(float f, Words a) {
  Words r;
  const float p = __fmul_rn(f, a.hi);
  r.hi = fast_two_sum(p, __fmaf_rn(f, a.lo, __fmaf_rn(f, a.hi, -p)), r.lo);
  return r;
}
__device__ __forceinline__ bool exceeds(Words a, Words b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

struct ExactWeight {
  float M;              // the largest logit, times `before`
  float before, after;  // powers of two for the logits and for their differences: temperatures of any size
  float c, cl;          // log2(e) / T, in two words
  const float2 *power;  // kPower32, where lanes read it side by side

  ExactWeight() = default;
  // T finite and > 0, M finite
  __device__ __forceinline__ ExactWeight(float m, float T, const float2 *p) {
    before = T > 0x1p64f ? 0x1p-64f : 1.f;
    after = T < 0x1p-64f ? 0x1p64f : 1.f;
    M = __fmul_rn(m, before);
    const float t = __fmul_rn(__fmul_rn(T, before), after);
    constexpr float hi = 0x1.715476p0f, lo = 0x1.4ae0cp-26f;  // log2(e)
    c = __fdiv_rn(hi, t);
    cl = __fdiv_rn(__fadd_rn(__fmaf_rn(-c, t, hi), lo), t);
    power = p;
  }
  // Weights of N pairs of logits that are finite or -inf and at most the largest; of
  // those below `floor` 0.  Some 40 instructions a pair and 8 a number, in a chain of 40:
  // several go through it side by side.  (fp64's exp would be some 30 of its own, each
  // as long as 60 of these.)
  template <int N>
  __device__ __forceinline__ void operator()(const float2 (&l)[N], float floor, float2 (&w)[N], float2 (&wl)[N]) const {
    float2 z[N], rest[N], t[N], p[N], pl[N];
    const bool scaled = before != 1.f || after != 1.f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float2 d, dl;
      if (scaled) {
        d = fmul2(two_sum(fmul2(l[n], both(before)), both(-M), dl), both(after));
        dl = fmul2(dl, both(after));
      } else {
        d = two_sum(l[n], both(-M), dl);
      }
      z[n] = fmul2(d, both(-c));  // -y, and what is left of y
      rest[n] = ffma2(d, both(cl), ffma2(dl, both(c), ffma2(d, both(c), z[n])));
      t[n] = minus2(both(0x1.8p18f), z[n]);  // to a 32nd: a sum of 1.5 2^18 has that unit
    }
    constexpr float hi = 0x1.62e43p-1f, lo = -0x1.05c61p-29f;  // ln 2
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float2 r = minus2(minus2(both(0x1.8p18f), t[n]), z[n]);
      const float2 x = fmul2(r, both(hi)), xl = ffma2(rest[n], both(hi), ffma2(r, both(lo), ffma2(r, both(hi), fmul2(x, both(-1.f)))));
      // e^(x + xl) - 1 = p + pl: x + x^2/2, and their rounding, x^3/6 and on, xl e^x
      const float2 q = fmul2(x, x);
      const float2 far = fmul2(fmul2(q, x), ffma2(x, ffma2(x, both(1.f / 120.f), both(1.f / 24.f)), both(1.f / 6.f)));
      p[n] = ffma2(q, both(0.5f), x);
      pl[n] = fadd2(ffma2(q, both(0.5f), minus2(x, p[n])), fadd2(far, ffma2(xl, p[n], xl)));
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i0 = __float_as_int(t[n].x) - __float_as_int(0x1.8p18f), i1 = __float_as_int(t[n].y) - __float_as_int(0x1.8p18f);
      const float2 u0 = power[i0 & 31], u1 = power[i1 & 31];
      const float2 u = make_float2(u0.x, u1.x), ul = make_float2(u0.y, u1.y);
      const float2 s = ffma2(u, p[n], u);
      const float2 sl = ffma2(u, pl[n], ffma2(ul, p[n], fadd2(ul, ffma2(u, p[n], minus2(u, s)))));
      const bool on0 = l[n].x >= floor && z[n].x < 126.f, on1 = l[n].y >= floor && z[n].y < 126.f;
      const float by0 = __int_as_float(((i0 >> 5) + 127) << 23), by1 = __int_as_float(((i1 >> 5) + 127) << 23);  // 2^-126 at least
      w[n] = make_float2(on0 ? __fmul_rn(s.x, by0) : 0.f, on1 ? __fmul_rn(s.y, by1) : 0.f);
      wl[n] = make_float2(on0 ? __fmul_rn(sl.x, by0) : 0.f, on1 ? __fmul_rn(sl.y, by1) : 0.f);
    }
  }
  __device__ __forceinline__ Words operator()(float l, float floor) const {
    const float2 pair[1] = {both(l)};
    float2 w[1], wl[1];
    (*this)(pair, floor, w, wl);
    return {w[0].x, wl[0].x};
  }
};

// Running sums of weights in two words, N pairs side by side, on top of 1: no weight is
// more, so that what a sum loses is got in two instructions.
template <int N>
struct ExactSum {
  float2 hi[N], lo[N];
  __device__ __forceinline__ ExactSum() {
#pragma unroll
    for (int n = 0; n < N; ++n) hi[n] = both(1.f), lo[n] = both(0.f);
  }
  __device__ __forceinline__ void add(const float2 (&w)[N], const float2 (&wl)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float2 s = fadd2(hi[n], w[n]);
      lo[n] = fadd2(lo[n], fadd2(fadd2(minus2(hi[n], s), w[n]), wl[n]));
      hi[n] = s;
    }
  }
  __device__ __forceinline__ Words all() const {
    Words s = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) s = add_words(add_words(s, {__fsub_rn(hi[n].x, 1.f), lo[n].x}), {__fsub_rn(hi[n].y, 1.f), lo[n].y});
    return s;
  }
};

}  // namespace sv
