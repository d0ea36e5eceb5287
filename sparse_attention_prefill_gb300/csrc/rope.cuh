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

// Thread t of a row and head (dim / 16 of them) has two units of 8 channels: with
// halves and t < rot / 16, channels 8 t.. and rot / 2 + 8 t.., whose pairs 8 t.. it
// rotates; otherwise 16 neighbouring ones.
struct Place {
  int a, b;                              // first channels of the units
  bool turns;                            // whether they are rotated, by pairs 8 t..
};
__device__ __forceinline__ Place place_of(int t, int rot, bool interleaved) {
  const bool turns = t < rot / 16;
  if (interleaved || !turns) return Place{16 * t, 16 * t + kUnit, turns};
  return Place{kUnit * t, rot / 2 + kUnit * t, true};
}

// cosines and sines of pairs 8 t .. 8 t + 7 at position p, times the amplitude
__device__ __forceinline__ void angles(const uint64_t *turn, int t, int64_t p, float amplitude,
                                       float sign, float (&c)[kUnit], float (&s)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    const uint64_t turns = (uint64_t)p * turn[kUnit * t + i];
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

// the 16 channels of a thread's two units; every product is rounded, so that a
// rotation has the same bits wherever it is computed
__device__ __forceinline__ void turn16(float (&x)[2 * kUnit], bool interleaved,
                                       const float (&c)[kUnit], const float (&s)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    float &a = interleaved ? x[2 * i] : x[i];
    float &b = interleaved ? x[2 * i + 1] : x[kUnit + i];
    const float u = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
    const float w = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
    a = u, b = w;
  }
}

}  // namespace rope
}  // namespace csa2
