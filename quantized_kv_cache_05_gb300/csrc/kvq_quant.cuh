// The quantizers' arithmetic shared by the append kernels: bf16 widening and
// the quotients whose E4M3 or E2M1 codes equal those of the IEEE division.
#pragma once

#include "kvq_device.cuh"

namespace kvq {

__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
}

// fl32(x_i / s) for a grid encoder whose rounding boundaries have at most
// 24 - log2(lowmask + 1) significant bits (E4M3: 5, lowmask 2^19 - 1; E2M1: 3,
// lowmask 2^21 - 1), for N elements.  With z = RN(1/s), q0 = RN(x z), r =
// RN(x - q0 s) and q = RN(q0 + r z) is within one fp32 step of RN(x/s) (the
// correction step of P. Markstein, IBM J. Res. Dev. 34(1), 1990).  Two
// adjacent fp32 numbers round to different codes only if one of them is a
// boundary, whose low fraction bits are zero; so where some q has low bits 0,
// 1 or all ones, ((bits + 1) & lowmask) <= 2 -- which also holds for
// infinities and the canonical NaN -- the IEEE division gives all N.  Either
// way every code equals the code of the correctly rounded quotient.
template <int N>
struct Floats {
  float v[N];
};

// The IEEE quotients of a whole group: out of line, so that the rarely taken
// fallback stays off the common path (not merged into it as predicated code).
template <int N>
__device__ __noinline__ Floats<N> ieee_quotients(Floats<N> x, float s) {
#pragma unroll
  for (int i = 0; i < N; ++i) x.v[i] = __fdiv_rn(x.v[i], s);
  return x;
}

template <int N>
__device__ __forceinline__ void quotients_for_codes(float (&x)[N], float s, float z,
                                                    uint32_t lowmask) {
  float q[N];
  uint32_t m = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float q0 = __fmul_rn(x[i], z);
    const float r = __fmaf_rn(-q0, s, x[i]);
    q[i] = __fmaf_rn(r, z, q0);
    m = min(m, (__float_as_uint(q[i]) + 1u) & lowmask);
  }
  if (m <= 2u) {
    Floats<N> in;
#pragma unroll
    for (int i = 0; i < N; ++i) in.v[i] = x[i];
    const Floats<N> out = ieee_quotients<N>(in, s);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = out.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = q[i];
  }
}

constexpr uint32_t kE4m3Low = (1u << 19) - 1;   // E4M3 boundaries: <= 5 significant bits
constexpr uint32_t kE2m1Low = (1u << 21) - 1;   // E2M1 boundaries: <= 3 significant bits

}  // namespace kvq
