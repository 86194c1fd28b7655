// Rotary positions: the angle of a (position, pair) and the rotation of the
// pairs that one thread holds. Shared by the rotation alone (k_rotary.cu) and
// the cache write (k_append.cu).
//
// Pair p of a head has the frequency f_p (fp32, radians per position) and is
// turned by theta = pos f_p:
//   y0 = A (x0 cos theta - x1 sin theta), y1 = A (x1 cos theta + x0 sin theta),
// elements (p, p + rot/2) of the head in the half layout, (2p, 2p + 1) in the
// interleaved one. The transpose (the backward pass) turns by -theta.
//
// theta reaches 5e5 radians at the end of a 512K context, where an fp32
// product is off by up to 0.03 radians. So the frequency is kept in turns as a
// 64-bit binary fraction, F = frac(f / 2 pi) 2^64: pos * F modulo 2^64 is the
// fraction of the last turn, wrapping exactly, and the error is that of F, two
// fp64 roundings and the fraction's last bit: 2^-52 f / 2 pi + 2^-64 turns a
// position (4e-11 turns at 2^20 positions and f = 1). The top bits give the nearest quarter turn, and all 64 an offset t
// of at most an eighth (pi/4 radians, kept to fp64's 53 bits, so that a sine or
// cosine near 0 is as exact as any other; 32 bits of it would be 1.5e-9 off), where
// the Taylor series of sin up to t^9 and of cos up
// to t^10 are within 2e-9 and 2e-10. They are summed in fp64 (a dozen
// operations at half the fp32 rate, half the instructions of two-part fp32
// sums) and rounded once, amplitude included: a bf16 key that lands on the
// other side of a rounding border moves its block's summary by far more than
// fp32 resolves, and every bit here halves how often.
#pragma once

#include <math.h>

#include "common.cuh"

namespace sas {

__device__ __forceinline__ unsigned long long turns_u64(float f) {
  const double t = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rd((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ void turn_sincos(unsigned long long F, int pos, float amp, float& c,
                                            float& s) {
  const unsigned long long ph = F * (unsigned long long)(long long)pos;
  const uint32_t quarter = ((uint32_t)(ph >> 32) + 0x20000000u) >> 30;  // nearest one (mod 4)
  // [-2^61, 2^61): an eighth of a turn, as the difference wraps
  const long long off = (long long)(ph - ((unsigned long long)quarter << 62));
  const double t = (double)off * (1.4629180792671596810513e-09 / 4294967296.0);  // 2 pi / 2^64
  const double q = t * t;
  const double sn =
      fma(t * q, fma(q, fma(q, fma(q, 1.0 / 362880, -1.0 / 5040), 1.0 / 120), -1.0 / 6), t);
  const double cs = fma(
      q, fma(q, fma(q, fma(q, fma(q, -1.0 / 3628800, 1.0 / 40320), -1.0 / 720), 1.0 / 24), -0.5), 1.0);
  const bool odd = quarter & 1u;
  const double a = amp;
  c = (float)((odd ? sn : cs) * ((quarter == 1u || quarter == 2u) ? -a : a));
  s = (float)((odd ? cs : sn) * ((quarter & 2u) ? -a : a));
}

// A thread holds units of 2 VN elements of a head: VN pairs. VN = Vec16<T>::N
// moves 16-byte vectors, VN = 1 single elements (rotated widths or strides that
// vectors do not fit).
// VN elements as they are stored. Loads are marked as read once (append, whose
// writes the next kernel reads, gains 5% from it).
template <typename T, int VN>
struct Piece {
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void unpack(float (&x)[VN]) const {
    Vec16<T>::load(reinterpret_cast<const T*>(&v), x);
  }
  __device__ __forceinline__ void pack(const float (&x)[VN]) {
    Vec16<T>::store(reinterpret_cast<T*>(&v), x);
  }
};
template <typename T>
struct Piece<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ void unpack(float (&x)[1]) const { x[0] = to_f(v); }
  __device__ __forceinline__ void pack(const float (&x)[1]) { v = from_f<T>(x[0]); }
};

// Where unit u (2 VN elements) of a head lies: its two element offsets.
// Units u < rot / (2 VN) are rotated, the others are passed through.
template <int VN>
__device__ __forceinline__ void unit_offsets(int u, int rot, bool interleaved, int& e0, int& e1) {
  const int ru = rot / (2 * VN);
  if (u < ru && !interleaved) {
    e0 = u * VN;
    e1 = (rot >> 1) + u * VN;
  } else {
    e0 = 2 * u * VN;
    e1 = e0 + VN;
  }
}

__device__ __forceinline__ void rotate_pair(float& x0, float& x1, float c, float s) {
  const float y0 = x0 * c - x1 * s, y1 = x1 * c + x0 * s;
  x0 = y0;
  x1 = y1;
}

// Rotates the VN pairs of (a, b): element i of a with element i of b (half
// layout), or neighbours within a, then within b (interleaved).
template <int VN>
__device__ __forceinline__ void rotate_unit(float (&a)[VN], float (&b)[VN], const float (&c)[VN],
                                            const float (&s)[VN], bool interleaved) {
  if (VN > 1 && interleaved) {
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      rotate_pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
      rotate_pair(b[2 * i], b[2 * i + 1], c[VN / 2 + i], s[VN / 2 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VN; ++i) rotate_pair(a[i], b[i], c[i], s[i]);
  }
}

// Turns per position of the VN pairs of rotated unit u: pairs u VN .. u VN +
// VN - 1 in both layouts. A frequency that is not finite has no turns: its bit
// of `bad` is set, and the pair's sine and cosine are NaN.
template <int VN>
struct UnitTurns {
  unsigned long long F[VN];
  uint32_t bad;

  __device__ __forceinline__ UnitTurns(const float* __restrict__ inv_freq, int u) : bad(0) {
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const float f = __ldg(inv_freq + u * VN + i);
      if (!(fabsf(f) < INFINITY)) bad |= 1u << i;
      F[i] = turns_u64(f);
    }
  }
  __device__ __forceinline__ void sincos(int pos, float amp, float (&c)[VN],
                                         float (&s)[VN]) const {
#pragma unroll
    for (int i = 0; i < VN; ++i) turn_sincos(F[i], pos, bad >> i & 1u ? NAN : amp, c[i], s[i]);
  }
};

}  // namespace sas
