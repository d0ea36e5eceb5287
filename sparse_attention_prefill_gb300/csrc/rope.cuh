// Rotary positions: what csa2_rotate and csa2_page_append share.
//
// A position p and a frequency f (radians per position) make p f / 2 pi turns, of
// which only the fraction counts.  A frequency is held as the fraction of a turn in
// units of 2^-64, so that p times it, modulo 2^64, is the fraction with no rounding
// but the frequency's own, 2^-64 of a turn at most: a product in fp32 would be a whole
// turn off at positions of 2^24, and one in fp64 costs its SM 32 cycles a warp.
#pragma once
#include "dense.cuh"

namespace csa2 {
namespace rope {

using dense::Elem;

constexpr int kUnit = 8;                 // channels of a 16-byte access

struct Rope {
  const double *freq;
  const int64_t *pos;
  int rot, interleaved;
  float amplitude;
};

inline int check_rope(const csa2_rope *r, int dim) {
  if (!r->freq) return CSA2_ERR_INVALID_ARG;
  if (!(r->amplitude - r->amplitude == 0.f)) return CSA2_ERR_INVALID_ARG;   // NaN, infinity
  if (r->rot < 16 || r->rot > dim || r->rot % 16) return CSA2_ERR_UNSUPPORTED;
  if (!aligned(8, r->freq, r->pos)) return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}

// The fraction of a turn that a frequency makes per position, in 2^-64, from its bits: the
// mantissa times 1 / 2 pi in 2^-128, shifted by the exponent (below 2^52).  (Times 1 / 2 pi
// in fp64 frequencies near 1 are 2^-56 of a turn off, which positions of 2^31 make 1.9e-7
// radians; with a second double for the rest a decode step's append takes 8.5 us instead of
// 7.9: fp64 is slow.)
__device__ __forceinline__ uint64_t turn_per_position(double freq) {
  constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;
  const uint64_t bits = (uint64_t)__double_as_longlong(freq);
  const uint64_t m = (bits & 0xfffffffffffffull) | (1ull << 52);     // times 2^(exponent - 1075)
  const uint64_t carry = __umul64hi(m, kLow), mid = m * kHigh + carry;
  const uint64_t high = __umul64hi(m, kHigh) + (mid < carry);
  const int right = 1011 - (int)((bits >> 52) & 0x7ff);
  const uint64_t t = right >= 0 ? high >> min(right, 63)             // (high has 51 bits)
                                : high << (-right & 63) | mid >> (right & 63);
  return bits >> 63 ? 0 - t : t;
}

// of the table's pairs, by a block
__device__ __forceinline__ void load_turns(const Rope &R, uint64_t *turn) {
  for (int i = threadIdx.x; i < R.rot / 2; i += blockDim.x) turn[i] = turn_per_position(R.freq[i]);
}

// Thread t of a row and head (dim / 16 of them) has two units of 8 channels, each
// unit's neighbours with the neighbouring threads.  Halves: with t < rot / 16, channels
// 8 t.. and rot / 2 + 8 t.., whose pairs it rotates; the others share out the channels
// behind.  Interleaved: channels 8 t.. and dim / 2 + 8 t.., four pairs each.
struct Place {
  int a, b;                              // first channels of the units
  bool ta, tb;                           // whether they are rotated
};
template <int D, bool kInterleaved>
__device__ __forceinline__ Place place_of(int t, int rot) {
  if (kInterleaved) return Place{kUnit * t, D / 2 + kUnit * t, kUnit * t < rot, D / 2 + kUnit * t < rot};
  const bool in = t < rot / 16;
  const int first = in ? kUnit * t : rot / 2 + kUnit * t;      // rot + 8 (t - rot / 16)
  return Place{first, first + (in ? rot : D - rot) / 2, in, in};
}

// amp * cos and amp * sin of a turn's fraction in 2^-64: off by 0.72 units of the last place
// (0.82 where there is an amplitude; the largest of ten million random turns), and near their
// zeros by 2^-48 of the amplitude, for 13 bits of the fraction that are cut off.
//
// The angle less quarter turns, within pi / 4, as a sum of two floats, then the Taylor sums
// (to a^9 and a^10: 3e-9 off) behind their leading terms a and 1 - a^2 / 2, which are kept
// with what their roundings lose.  (Without an amplitude the result is that of 64 bits,
// rounded once, in 98 cases of a hundred: an 8-bit code then hardly ever depends on who
// rotated.)
__device__ __forceinline__ void turn_of(uint64_t turn, float amp, float &c, float &s) {
  const uint32_t q = (uint32_t)((turn + (1ull << 61)) >> 62);
  const int64_t r = (int64_t)(turn - ((uint64_t)q << 62));
  const float h = (float)(int32_t)(r >> 37) * 0x1p-27f;          // both exact
  const float l = (float)(int32_t)(((uint64_t)r >> 13) & 0xffffffu) * 0x1p-51f;
  constexpr float kTwoPi = 6.2831854820251465f, kRest = -1.7484555e-7f;
  const float a = h * kTwoPi;
  const float al = fmaf(l, kTwoPi, fmaf(h, kRest, fmaf(h, kTwoPi, -a)));
  const float z = a * a, zl = fmaf(a, a, -z);
  const float ps =
      fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6);
  const float pc =
      fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24);
  float lo[2], hi[2];                    // cosine, sine
  hi[0] = fmaf(-0.5f, z, 1.f);
  lo[0] = fmaf(z * z, pc, fmaf(-a, al, fmaf(-0.5f, zl, fmaf(-0.5f, z, 1.f - hi[0]))));
  hi[1] = a;
  lo[1] = fmaf(a * z, ps, fmaf(-0.5f * z, al, al));
  float v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float p = hi[i] * amp;
    v[i] = p + fmaf(lo[i], amp, fmaf(hi[i], amp, -p));
  }
  const float x = q & 1 ? v[1] : v[0], y = q & 1 ? v[0] : v[1];
  c = (q + 1) & 2 ? -x : x;
  s = q & 2 ? -y : y;
}

// cosines and sines of a thread's pairs at position p, times the amplitude
template <int D, bool kInterleaved>
__device__ __forceinline__ void angles(const uint64_t *turn, int t, const Place &at, int64_t p,
                                       float amplitude, float sign, float (&c)[kUnit],
                                       float (&s)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    if (i < kUnit / 2 ? !at.ta : !at.tb) continue;
    const int pair = !kInterleaved     ? kUnit * t + i
                     : i < kUnit / 2 ? kUnit / 2 * t + i
                                     : D / 4 + kUnit / 2 * (t - 1) + i;
    turn_of((uint64_t)p * turn[pair], amplitude, c[i], s[i]);
    s[i] *= sign;
  }
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if (Elem<T>::kBf16) {
      f.x = __uint_as_float(v[i] << 16);
      f.y = __uint_as_float(v[i] & 0xffff0000u);
    } else {
      f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
    }
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// the 16 channels of a thread's two units; every product is rounded, so that a
// rotation has the same bits wherever it is computed
template <bool kInterleaved>
__device__ __forceinline__ void turn16(float (&x)[2 * kUnit], const Place &at,
                                       const float (&c)[kUnit], const float (&s)[kUnit]) {
  using dense::add2;
  using dense::pack2;
  using dense::unpack2;
  if constexpr (!kInterleaved) {         // two pairs at a time
    if (!at.ta) return;
#pragma unroll
    for (int i = 0; i < kUnit; i += 2) {
      const uint64_t a = pack2(x[i], x[i + 1]), b = pack2(x[kUnit + i], x[kUnit + i + 1]);
      const uint64_t co = pack2(c[i], c[i + 1]), si = pack2(s[i], s[i + 1]);
      const float2 u = unpack2(sub2(mul2(a, co), mul2(b, si)));
      const float2 w = unpack2(add2(mul2(b, co), mul2(a, si)));
      x[i] = u.x, x[i + 1] = u.y, x[kUnit + i] = w.x, x[kUnit + i + 1] = w.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      if (i < kUnit / 2 ? !at.ta : !at.tb) continue;
      float &a = x[2 * i], &b = x[2 * i + 1];
      const float u = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
      const float w = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
      a = u, b = w;
    }
  }
}

}  // namespace rope
}  // namespace csa2
