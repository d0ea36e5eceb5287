// Rotary positions: what csa2_rotate and csa2_page_append share.
//
// A position p and a frequency f (radians per position) make p f / 2 pi turns, of
// which only the fraction counts.  A frequency is held as the fraction of a turn in
// units of 2^-64, so that p times it, modulo 2^64, is the fraction with no rounding
// but the frequency's own 2^-65: a product in fp32 would be a whole turn off at
// positions of 2^24, and one in fp64 costs its SM 32 cycles a warp.
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

// fractions of a turn per position, in 2^-64, of the table's pairs, by a block
__device__ __forceinline__ void load_turns(const Rope &R, uint64_t *turn) {
  for (int i = threadIdx.x; i < R.rot / 2; i += blockDim.x) {
    double t = R.freq[i] * 0.15915494309189535;     // 1 / 2 pi
    t -= floor(t);
    turn[i] = __double2ull_rn(t * 18446744073709551616.0);
  }
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
    const uint64_t turns = (uint64_t)p * turn[pair];
    // half turns from -1 to 1, to 2^-24
    const float x = (float)(int32_t)(turns >> 32) * 0x1p-31f;
    float si, co;
    sincospif(x, &si, &co);
    c[i] = co * amplitude;
    s[i] = si * amplitude * sign;
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
      const uint64_t co = pack2(c[i], c[i + 1]);
      const float2 u = unpack2(add2(mul2(a, co), mul2(b, pack2(-s[i], -s[i + 1]))));
      const float2 w = unpack2(add2(mul2(b, co), mul2(a, pack2(s[i], s[i + 1]))));
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
