// Per-head RMS norm and position rotation of queries and keys, and the append
// that applies them on the way into the paged cache (sm_103a).
//
// For one head x of D elements, all in fp32 from the bf16 input:
//   n_i = (x_i r) w_i,  r = 1 / sqrt(sum x^2 / D + eps)          (optional norm)
//   (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin)          (rotation)
// over the pairs (i, i + rot/2) or (2i, 2i + 1) of the first rot elements, the
// cosines and sines of the token's position read from the caller's fp32 table;
// the rest of the head passes unrotated.  Queries leave as bf16 or as E4M3
// codes, keys as bf16 rows or, in the append, as cache codes with the
// arithmetic of the plain append (one rounding of the fp32 value either way).
//
// Bound by HBM (2 bytes in, 1 or 2 out per element) for chunks and by the
// launch for decode steps.  D / 16 lanes share a row, each with two 8-element
// pieces: in the rotated part piece p and the piece rot/2 elements further on,
// which hold both members of eight pairs of the half-split order, so that no
// value moves between lanes (pairs side by side lie within a piece anyway).
// Both 16-byte loads of a lane group cover whole 32-byte sectors, the row's sum
// of squares is a butterfly over its lanes, and an NVFP4 block of 16 is the
// pieces of two neighbouring lanes (rot is a multiple of 32).  The arithmetic
// runs on packed fp32 pairs.
//
// Measured on GB300: 8192 tokens x 40 heads of 128 with norm, bf16 out (172 MB):
// 30.2 us, 5.7 TB/s, 85% of the copy rate; one token each of 64 requests: 2.3
// us, where an empty kernel takes 0.7: the latency of its loads one behind the
// other.  The append of 4 x 2048 ragged padded tokens (48 heads, 94 MB): 27.0 us,
// 52% of the copy rate; 57 to 62% of the issue slots while an SM is busy, 46% over
// the kernel.  One token each of 48 requests: 4.3 us.  Settling quotients takes
// 0.8 and 0.7 us of these two.  The packed append of 8000 tokens (48 heads, 184 MB): 45.0
// us, 60% of the copy rate; 63% of the issue slots while an SM is busy, no pipe full, with 5.3
// warps a scheduler.

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

// Small blocks, so that the last ones to run leave few SMs idle (the append of
// 4 x 2048 padded tokens, 48 heads: 26.4 us against 27.3 with half as many of
// 256 threads), six to an SM: with four 29.1 us, with eight, which leave 64
// registers, 28.1.  Rows that leave as bf16 take 30 us with either (8192 tokens,
// 40 heads).
constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 6;
// From this many lanes (two thousand per SM) on, groups take kRowsEach rows: the
// append of 4 x 2048 padded tokens takes 26.5 us so against 47.0 with a group for
// every row (three rows each: 29.4, twelve: 27.0).  Fewer lanes than that fill the
// GPU only once.
constexpr unsigned long long kManyThreads = 152ull * 2048;
constexpr int kRowsEach = 6;

// The two pieces (8 elements each) of lane p of a row of D elements, the first
// `rot` of them rotated.
struct Pieces {
  int c0, c1;
  bool turn;
};
template <int D>
__device__ __forceinline__ Pieces pieces(int p, int rot) {
  const int nr = rot / 16;   // lanes that hold rotated pieces
  Pieces r;
  r.turn = p < nr;
  r.c0 = r.turn ? p : p + nr;
  r.c1 = r.c0 + (r.turn ? nr : D / 16 - nr);
  return r;
}

// A lane's 16 elements as packed pairs: v[0..3] its first piece, v[4..7] its second.
struct Row {
  uint64_t v[8];

  static __device__ __forceinline__ uint64_t widen(uint32_t w) {   // two bf16
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ __forceinline__ void from_bf16(uint4 x0, uint4 x1) {
    v[0] = widen(x0.x); v[1] = widen(x0.y); v[2] = widen(x0.z); v[3] = widen(x0.w);
    v[4] = widen(x1.x); v[5] = widen(x1.y); v[6] = widen(x1.z); v[7] = widen(x1.w);
  }
  static __device__ __forceinline__ uint32_t narrow(uint64_t p) {
    const float2 f = unpack2(p);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ void store_bf16(uint16_t* row, const Pieces& pc) const {
    *reinterpret_cast<uint4*>(row + 8 * pc.c0) =
        make_uint4(narrow(v[0]), narrow(v[1]), narrow(v[2]), narrow(v[3]));
    *reinterpret_cast<uint4*>(row + 8 * pc.c1) =
        make_uint4(narrow(v[4]), narrow(v[5]), narrow(v[6]), narrow(v[7]));
  }
  // RMS norm of a row spread over LANES lanes: r here (every lane of the warp
  // calls it; the length is a power of two), the weights below.
  template <int LANES>
  __device__ __forceinline__ float inv_rms(float eps) const {
    uint64_t s2 = 0ull;
#pragma unroll
    for (int i = 0; i < 8; ++i) s2 = fma2(v[i], v[i], s2);
    const float2 s = unpack2(s2);
    float ss = s.x + s.y;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // the approximate root and one correction step: within half a unit or so,
    // where the approximation alone would add most of the row's error (codes
    // next to a rounding boundary feel it)
    const float x = ss * (1.0f / (LANES * 16)) + eps, r = rsqrtf(x);
    const float e = __fmaf_rn(-__fmul_rn(x, r), r, 1.f);
    return fabsf(e) < 1.f ? __fmaf_rn(0.5f * r, e, r) : r;   // (not at 0, infinity, NaN)
  }
  __device__ __forceinline__ void norm(float r, const float* w, const Pieces& pc) {
    const uint64_t r2 = pack2(r, r);
    const float4* w0 = reinterpret_cast<const float4*>(w + 8 * pc.c0);
    const float4* w1 = reinterpret_cast<const float4*>(w + 8 * pc.c1);
    const float4 a = __ldg(w0), b = __ldg(w0 + 1), c = __ldg(w1), d = __ldg(w1 + 1);
    v[0] = mul2(mul2(v[0], r2), pack2(a.x, a.y));
    v[1] = mul2(mul2(v[1], r2), pack2(a.z, a.w));
    v[2] = mul2(mul2(v[2], r2), pack2(b.x, b.y));
    v[3] = mul2(mul2(v[3], r2), pack2(b.z, b.w));
    v[4] = mul2(mul2(v[4], r2), pack2(c.x, c.y));
    v[5] = mul2(mul2(v[5], r2), pack2(c.z, c.w));
    v[6] = mul2(mul2(v[6], r2), pack2(d.x, d.y));
    v[7] = mul2(mul2(v[7], r2), pack2(d.z, d.w));
  }
};

// The angles of a lane's eight pairs, and the rotation of its elements.
// Half-split order: both members of a pair lie at the same place in the two
// pieces; side by side (INTER): in the two halves of a packed pair, which takes
// the cosine (sine) twice.
template <bool INTER>
struct Angles {
  static constexpr int kN = INTER ? 8 : 4;
  uint64_t c[kN], s[kN], n[INTER ? 1 : kN];   // cos, sin (INTER: (-sin, sin)), -sin
  // trow: the position's cosines, then (half further on) its sines
  __device__ __forceinline__ void load(const float* trow, int half, const Pieces& pc) {
    const int i0 = INTER ? 4 * pc.c0 : 8 * pc.c0, i1 = INTER ? 4 * pc.c1 : 8 * pc.c0 + 4;
    const float4 ca = __ldg(reinterpret_cast<const float4*>(trow + i0));
    const float4 cb = __ldg(reinterpret_cast<const float4*>(trow + i1));
    const float4 sa = __ldg(reinterpret_cast<const float4*>(trow + half + i0));
    const float4 sb = __ldg(reinterpret_cast<const float4*>(trow + half + i1));
    const float cs[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
    const float sn[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if constexpr (INTER) {
        c[i] = pack2(cs[i], cs[i]);
        s[i] = pack2(-sn[i], sn[i]);
      } else {
        c[i] = pack2(cs[2 * i], cs[2 * i + 1]);
        s[i] = pack2(sn[2 * i], sn[2 * i + 1]);
        n[i] = pack2(-sn[2 * i], -sn[2 * i + 1]);
      }
    }
  }
  __device__ __forceinline__ void apply(Row& x) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if constexpr (INTER) {
        const float2 f = unpack2(x.v[i]);
        x.v[i] = fma2(x.v[i], c[i], mul2(pack2(f.y, f.x), s[i]));
      } else {
        const uint64_t a = x.v[i], b = x.v[4 + i];
        x.v[i] = fma2(a, c[i], mul2(b, n[i]));
        x.v[4 + i] = fma2(b, c[i], mul2(a, s[i]));
      }
    }
  }
};

__device__ __forceinline__ uint2 pack_e4m3x8(const float* f) {
  const uint32_t lo = f32x2_to_e4m3x2(f[0], f[1]) | (f32x2_to_e4m3x2(f[2], f[3]) << 16);
  const uint32_t hi = f32x2_to_e4m3x2(f[4], f[5]) | (f32x2_to_e4m3x2(f[6], f[7]) << 16);
  return make_uint2(lo, hi);
}

// Sums of two fp32 numbers, hi + lo: some 48 bits from the exact errors of sums
// (D. Knuth, The Art of Computer Programming 2, 4.2.2) and of fused products.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Pair times(Pair a, Pair b) {
  Pair p = two_prod(a.hi, b.hi);
  p.lo += __fmaf_rn(a.hi, b.lo, a.lo * b.hi);
  return p;
}
__device__ __forceinline__ Pair plus(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;
}

// 1 / rms of a row spread over LANES lanes as a pair (every lane of the warp
// calls it).  One step of correction leaves 3/8 e^2 of it, e = 1 - v r^2 with the
// approximate root: 2^-43 where that is off by its two units.
template <int LANES>
__device__ __forceinline__ Pair inv_rms_pair(const Row& x, float eps) {
  Pair s = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack2(x.v[i]);
    // squares of bf16 values are exact
    Pair t = two_sum(s.hi, __fmul_rn(f.x, f.x));
    s.lo += t.lo;
    t = two_sum(t.hi, __fmul_rn(f.y, f.y));
    s = {t.hi, s.lo + t.lo};
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    s = plus(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
  constexpr float kMean = 1.0f / (LANES * 16);   // a power of two
  const Pair v = plus({s.hi * kMean, s.lo * kMean}, {eps, 0.f});
  const float r = rsqrtf(v.hi);
  const Pair rr = two_prod(r, r);
  const float e =
      __fmaf_rn(-v.hi, rr.hi, 1.f) - __fmaf_rn(v.hi, rr.lo, v.lo * rr.hi);   // 1 - v r^2
  return {r, fabsf(e) < 1.f ? 0.5f * r * e : 0.f};   // (not at 0, infinity, NaN)
}

// Whether a quotient lies within `near` fp32 steps of an E4M3 rounding boundary
// (their low 19 fraction bits are zero).
__device__ __forceinline__ bool near_boundary(float q, uint32_t near) {
  return ((__float_as_uint(q) + near) & kE4m3Low) <= 2 * near;
}

// Of a lane's 16 quotients, those next to a rounding boundary moved to the side
// of it (or onto it) where y / s lies with y from the formulas in pairs: so
// close, the fp32 steps before the quotient could decide the code.  The
// arguments one by one: they stay in registers.  x, w: the head's row and its
// weights (or null); r: hi + lo of its 1 / rms.
template <bool INTER>
__device__ __noinline__ Floats<16> settle(Floats<16> q, const uint16_t* x, const float* w,
                                          const float* trow, int half, float r_hi, float r_lo,
                                          int c0, int c1, bool turn, float s, uint32_t near) {
  auto value = [&](int i) -> Pair {
    const float v = bf16_bits_to_f32(x[i]);
    return w ? times(two_prod(v, w[i]), {r_hi, r_lo}) : Pair{v, 0.f};
  };
  auto side = [&](float f, Pair y) -> float {
    if (!near_boundary(f, near) || !(fabsf(f) < 1000.f)) return f;   // (480 is the last boundary)
    const uint32_t bits = __float_as_uint(f) & 0x7FFFFFFFu;
    const uint32_t b = (bits + (1u << 18)) & ~kE4m3Low;   // the boundary next to |f|
    const Pair bs = two_prod(__uint_as_float(b), s);
    const float sign = f < 0.f ? -1.f : 1.f;
    const float d = (sign * y.hi - bs.hi) + (sign * y.lo - bs.lo);   // (|y| - b s: hi - hi is exact)
    const uint32_t to = d > 0.f ? b + 1 : (d < 0.f && b > 0) ? b - 1 : b;
    return __uint_as_float(to | (__float_as_uint(f) & 0x80000000u));
  };
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    // the lane's pair k (rotated or not)
    const int ka = INTER ? 2 * k : k, kb = INTER ? 2 * k + 1 : 8 + k;
    if (!near_boundary(q.v[ka], near) && !near_boundary(q.v[kb], near)) continue;
    const int ia = 8 * (ka < 8 ? c0 : c1) + (ka & 7), ib = 8 * (kb < 8 ? c0 : c1) + (kb & 7);
    Pair a = value(ia), b = value(ib);
    if (turn) {
      const int t = INTER ? ia / 2 : ia;
      const Pair c = {trow[t], 0.f}, sn = {trow[half + t], 0.f}, nsn = {-trow[half + t], 0.f};
      const Pair a0 = a;
      a = plus(times(a0, c), times(b, nsn));
      b = plus(times(b, c), times(a0, sn));
    }
    q.v[ka] = side(q.v[ka], a);
    q.v[kb] = side(q.v[kb], b);
  }
  return q;
}

// E4M3(fl32(x / s)) of a lane's 16 elements (z = RN(1/s)): the quotients of
// quotients_for_codes, in packed pairs.  Where one lies within `near` fp32 steps
// of a rounding boundary, `exact` settles them: by the IEEE division of what came
// in as it is (near = 1), or by `settle` for what was computed in fp32.
template <typename F>
__device__ __forceinline__ void store_e4m3(const Row& x, float s, float z, uint8_t* row,
                                           const Pieces& pc, uint32_t near, F&& exact) {
  const uint64_t z2 = pack2(z, z), ns2 = pack2(-s, -s);
  Floats<16> q;
  uint32_t m = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t q0 = mul2(x.v[i], z2);
    const float2 f = unpack2(fma2(fma2(q0, ns2, x.v[i]), z2, q0));
    q.v[2 * i] = f.x;
    q.v[2 * i + 1] = f.y;
    m = min(m, min((__float_as_uint(f.x) + near) & kE4m3Low, (__float_as_uint(f.y) + near) & kE4m3Low));
  }
  if (m <= 2 * near) q = exact(q);
  *reinterpret_cast<uint2*>(row + 8 * pc.c0) = pack_e4m3x8(q.v);
  *reinterpret_cast<uint2*>(row + 8 * pc.c1) = pack_e4m3x8(q.v + 8);
}

// Steps of a computed quotient from a boundary (or a grid value: both have zeros in
// their low bits) within which it is settled in pairs, 33 of 2^19: fp32's error is 2
// to 3 steps as a rule, 2 u of the rotation's larger product without a norm and 12.5
// u with one at most.
constexpr uint32_t kNear = 16;

// One NVFP4 half block (8 elements; the neighbouring lane holds the other
// half): codes in a word, and the block's scale code.  Every lane of the warp
// calls it.
__device__ __forceinline__ uint32_t nvfp4_half(const uint64_t* v, float g, uint32_t& sc) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2(v[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
  float bamax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) bamax = fmaxf(bamax, fabsf(f[i]));
  bamax = fmaxf(bamax, __shfl_xor_sync(0xffffffffu, bamax, 1));
  const float scf = __fdiv_rn(__fdiv_rn(bamax, 6.0f), g);
  sc = f32x2_to_e4m3x2(scf, 0.f) & 0xFFu;
  const float es = __fmul_rn(unpack_f16x2(e4m3x2_to_f16x2(sc)).x, g);
  if (es == 0.f) return 0u;
  quotients_for_codes<8>(f, es, __frcp_rn(es), kE2m1Low);
  return f32x8_to_e2m1x8(f);
}

// Both pieces of a lane as NVFP4 codes of cache row `row`; `ok` gates the stores.
template <int D>
__device__ __forceinline__ void store_nvfp4(const Row& x, float g, bool ok, uint8_t* codes,
                                            uint8_t* scales, long row, const Pieces& pc) {
  uint32_t s0, s1;
  const uint32_t w0 = nvfp4_half(x.v, g, s0), w1 = nvfp4_half(x.v + 4, g, s1);
  if (!ok) return;
  *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + 4 * pc.c0) = w0;
  *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + 4 * pc.c1) = w1;
  if ((pc.c0 & 1) == 0) {
    scales[row * (D / 16) + (pc.c0 >> 1)] = (uint8_t)s0;
    scales[row * (D / 16) + (pc.c1 >> 1)] = (uint8_t)s1;
  }
}

// Position and request of a token.  A token takes no part (nothing of it is
// read or written) when it lies past its request's new tokens, at a negative
// position, or -- which sets an error bit -- at a position past the table.
struct Token {
  int b;
  long pos;
  bool ok;
};
__device__ __forceinline__ Token token_of(const RopeArgs& a, unsigned token, bool report) {
  Token k;
  k.ok = true;
  k.b = 0;
  if (a.start_pos) {
    k.b = (int)(token / (unsigned)a.T);
    const int t = (int)(token - (unsigned)k.b * (unsigned)a.T);
    if (a.new_lens && t >= __ldg(a.new_lens + k.b)) k.ok = false;
    k.pos = (long)__ldg(a.start_pos + k.b) + t;
  } else {
    k.pos = a.positions ? __ldg(a.positions + token) : 0;
  }
  if (k.pos < 0) k.ok = false;
  if (k.ok && a.rot > 0 && k.pos >= a.num_positions) {
    k.ok = false;
    if (report) record_error(a.error_flag, 8);
  }
  return k;
}

// Cache row of kv head 0 at the token's position (head h: + h page_size), or -1
// (skipped): past the block table as in the plain append, or a page index out
// of range.  In a packed step (SLOTS) the token's slot says it: below zero, or past the
// cache, skipped.
template <bool SLOTS>
__device__ __forceinline__ long rope_page(const RopeArgs& a, const Token& k, unsigned token,
                                          bool report) {
  if constexpr (SLOTS) {
    const long slot = __ldg(a.slots + token);
    if (slot < 0) return -1;
    if (slot >= (long)a.num_pages * a.ps) {   // (below 2^31, as the cache's rows are)
      if (report) record_error(a.error_flag, 4);
      return -1;
    }
    const unsigned page = (unsigned)slot / (unsigned)a.ps;
    return (long)page * a.Hkv * a.ps + ((unsigned)slot - page * (unsigned)a.ps);
  } else {
    if (k.pos >= (long)a.max_pages * a.ps) return -1;
    const unsigned pos = (unsigned)k.pos, pi = pos / (unsigned)a.ps;
    const int page = __ldg(a.block_table + (size_t)k.b * a.max_pages + pi);
    if (page < 0 || page >= a.num_pages) {
      if (report) record_error(a.error_flag, 4);
      return -1;
    }
    return (long)page * a.Hkv * a.ps + (pos - pi * (unsigned)a.ps);
  }
}

// FMT 0: bf16 rows out (kvq_norm_rope); otherwise K and V go to the cache.
// `per_token` lane groups of a block share a token (a power of two), and
// gridDim.y blocks: a group takes every (per_token gridDim.y)-th of the token's
// rows (queries, keys, values in one numbering), the next row's loads going
// out before the present one's arithmetic.
// QF8 (FMT 0): the queries leave as E4M3 codes.  SLOTS: see rope_page (a variant: decided at
// run time it costs the append of 48 single tokens 0.06 us of 3.70).
template <int D, int FMT, bool INTER, bool QF8, bool SLOTS>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_kernel(const RopeArgs a, int per_token) {
  // the append is an ordinary launch (it starts after all earlier work), the
  // other a programmatic one
  if constexpr (FMT == 0) griddep_wait();
  griddep_launch_dependents();
  constexpr int kLanes = D / 16, kGroups = kRopeThreads / kLanes;
  const int p = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const unsigned token = blockIdx.x * (unsigned)(kGroups / per_token) + group / per_token;
  const bool q_codes = FMT == 0 ? QF8 : a.q_fp8 != 0;
  const int nq = a.q.heads, nqk = nq + a.k.heads, H = nqk + (FMT == 0 ? 0 : a.v.heads);
  const int first = blockIdx.y * per_token + group % per_token, step = per_token * gridDim.y;
  const bool in = token < a.tokens, report = in && p == 0 && first == 0;
  const Token tk = token_of(a, in ? token : 0, report);
  const bool ok = in && tk.ok;
  if (!__any_sync(0xffffffffu, ok)) return;   // padding: the whole warp
  const Pieces turned = pieces<D>(p, a.rot);

  auto fetch = [&](int i, uint4& x0, uint4& x1) {
    x0 = x1 = make_uint4(0, 0, 0, 0);
    if (!ok || i >= H) return;
    const bool isq = i < nq, isv = FMT != 0 && i >= nqk;
    const RopeRows& src = isq ? a.q : isv ? a.v : a.k;
    const int h = i - (isq ? 0 : isv ? nqk : nq);
    const uint16_t* x = src.data + (long)token * src.token_stride + (long)h * src.head_stride;
    const Pieces pc = isv ? pieces<D>(p, 0) : turned;
    x0 = *reinterpret_cast<const uint4*>(x + 8 * pc.c0);
    x1 = *reinterpret_cast<const uint4*>(x + 8 * pc.c1);
  };
  uint4 x0, x1;
  fetch(first, x0, x1);
  Angles<INTER> ang;
  if (turned.turn && ok) ang.load(a.cos_sin + tk.pos * a.rot, a.rot / 2, turned);
  // cache row of kv head 0: the token's, whatever the head
  long page_row = -1;
  if constexpr (FMT != 0) page_row = ok ? rope_page<SLOTS>(a, tk, token, report) : -1;

#pragma unroll 1
  for (int i0 = 0; i0 < H; i0 += step) {   // the same rounds for every lane of the warp
    const int i = i0 + first;
    const bool row = ok && i < H;
    const bool isq = i < nq, isv = FMT != 0 && i >= nqk;
    const int h = i - (isq ? 0 : isv ? nqk : nq);
    const Pieces pc = isv ? pieces<D>(p, 0) : turned;
    Row f;
    f.from_bf16(x0, x1);
    if (i0 + step < H) fetch(i + step, x0, x1);
    // every lane of the warp takes part in the norm's butterfly when any row
    // of the call has a norm
    const float* w = isq ? a.q_norm : isv ? nullptr : a.k_norm;
    Pair r = {1.f, 0.f};
    if (a.q_norm || a.k_norm) {
      const bool coded = w && (isq ? q_codes : FMT == kFmtFp8);
      if ((FMT != 0 || QF8) && __any_sync(0xffffffffu, coded))
        r = inv_rms_pair<kLanes>(f, a.eps);
      else
        r.hi = f.template inv_rms<kLanes>(a.eps);
      if (w) f.norm(r.hi + r.lo, w, pc);
    }
    if (turned.turn && !isv) ang.apply(f);

    // E4M3 codes: values that are the input itself take the plain append's
    // quotient, computed ones next to a rounding boundary are settled
    const bool computed = w != nullptr || (pc.turn && !isv);
    auto codes_to = [&](float s, float z, uint8_t* to) {
      store_e4m3(f, s, z, to, pc, computed ? kNear : 1u, [&](const Floats<16>& q) -> Floats<16> {
        if (computed) {
          const RopeRows& src = isq ? a.q : a.k;
          return settle<INTER>(q, src.data + (long)token * src.token_stride + (long)h * src.head_stride,
                               w, a.cos_sin + tk.pos * a.rot, a.rot / 2, r.hi, r.lo, pc.c0, pc.c1,
                               pc.turn, s, kNear);
        }
        Floats<16> in;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 v = unpack2(f.v[k]);
          in.v[2 * k] = v.x;
          in.v[2 * k + 1] = v.y;
        }
        return ieee_quotients<16>(in, s);
      });
    };

    if (isq || FMT == 0) {
      if (row) {
        const RopeRows& dst = isq ? a.q_out : a.k_out;
        const long at = (long)token * dst.token_stride + (long)h * dst.head_stride;
        if (isq && q_codes) {
          const float s = a.q_hs ? __ldg(a.q_hs + h) : a.q_scale;
          codes_to(s, a.q_hs ? __frcp_rn(s) : a.q_recip, reinterpret_cast<uint8_t*>(dst.data) + at);
        } else {
          f.store_bf16(dst.data + at, pc);
        }
      }
    }
    if constexpr (FMT != 0) {
      const bool store = row && !isq && page_row >= 0;
      const long crow = page_row + (long)h * a.ps;
      const float* hs = isv ? a.v_hs : a.k_hs;
      const float s = (hs && store) ? __ldg(hs + h) : (isv ? a.v_scale : a.k_scale);
      uint8_t* codes = isv ? a.v_codes : a.k_codes;
      if constexpr (FMT == kFmtFp8) {
        if (store)
          codes_to(s, hs ? __frcp_rn(s) : (isv ? a.v_recip : a.k_recip), codes + crow * D);
      } else {   // lanes without a row stay for their neighbours' shuffles
        store_nvfp4<D>(f, s, store, codes, isv ? a.v_bscale : a.k_bscale, crow, pc);
      }
    }
  }
}

// MLA: one warp per token, the 512-wide latent (normed, then NVFP4) on all
// lanes, the 64 rope-key elements (rotated, bf16) on the first four.
template <bool INTER, bool SLOTS>
__global__ void __launch_bounds__(kRopeThreads) rope_mla_kernel(const RopeArgs a) {
  griddep_launch_dependents();
  constexpr int D = 512, kRope = 64;
  const int lane = threadIdx.x & 31;
  const unsigned token = blockIdx.x * (unsigned)(kRopeThreads / 32) + threadIdx.x / 32;
  if (token >= a.tokens) return;   // the whole warp, as below
  const Token tk = token_of(a, token, lane == 0);
  const long crow = tk.ok ? rope_page<SLOTS>(a, tk, token, lane == 0) : -1;
  if (crow < 0) return;

  const Pieces pc = pieces<D>(lane, 0);
  const uint16_t* x = a.k.data + (long)token * a.k.token_stride;
  const uint4 x0 = *reinterpret_cast<const uint4*>(x + 8 * pc.c0);
  const uint4 x1 = *reinterpret_cast<const uint4*>(x + 8 * pc.c1);
  uint4 e0 = make_uint4(0, 0, 0, 0), e1 = e0;
  const Pieces pe = pieces<kRope>(lane & 3, a.rot);
  const uint16_t* xe = a.v.data + (long)token * a.v.token_stride;
  if (lane < kRope / 16) {
    e0 = *reinterpret_cast<const uint4*>(xe + 8 * pe.c0);
    e1 = *reinterpret_cast<const uint4*>(xe + 8 * pe.c1);
  }
  Row f;
  f.from_bf16(x0, x1);
  if (a.k_norm) f.norm(f.inv_rms<32>(a.eps), a.k_norm, pc);
  store_nvfp4<D>(f, a.k_scale, true, a.k_codes, a.k_bscale, crow, pc);
  if (lane < kRope / 16) {
    f.from_bf16(e0, e1);
    if (pe.turn) {
      Angles<INTER> ang;
      ang.load(a.cos_sin + tk.pos * a.rot, a.rot / 2, pe);
      ang.apply(f);
    }
    f.store_bf16(a.k_pe + crow * kRope, pe);
  }
}

template <int D, bool INTER>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  constexpr int kGroups = kRopeThreads / (D / 16);
  const int H = a.q.heads + a.k.heads + a.v.heads;
  // Few tokens: a group for every row, so that all loads go out at once.  Many:
  // fewer groups per token, which keep its angles, page and place for several
  // rows.
  int per_token = kGroups;
  while (per_token > 1 && per_token >= 2 * H) per_token /= 2;
  unsigned y = (unsigned)std::min((H + per_token - 1) / per_token, 65535);
  const unsigned long long threads = (unsigned long long)a.tokens * (D / 16);
  if (threads * H >= kManyThreads) {
    while (per_token > 1 && threads * per_token >= kManyThreads && per_token * kRowsEach > H)
      per_token /= 2;
    y = 1;
  }
  const unsigned per_block = (unsigned)(kGroups / per_token);
  const dim3 grid((a.tokens + per_block - 1) / per_block, y), block(kRopeThreads);
  if (a.fmt == 0 && a.q_fp8)
    return launch_pdl(rope_kernel<D, 0, INTER, true, false>, grid, block, 0, st, a, per_token);
  if (a.fmt == 0)
    return launch_pdl(rope_kernel<D, 0, INTER, false, false>, grid, block, 0, st, a, per_token);
  if (a.fmt == kFmtFp8 && a.slots)
    rope_kernel<D, kFmtFp8, INTER, false, true><<<grid, block, 0, st>>>(a, per_token);
  else if (a.fmt == kFmtFp8)
    rope_kernel<D, kFmtFp8, INTER, false, false><<<grid, block, 0, st>>>(a, per_token);
  else if (a.slots)
    rope_kernel<D, kFmtNvfp4, INTER, false, true><<<grid, block, 0, st>>>(a, per_token);
  else
    rope_kernel<D, kFmtNvfp4, INTER, false, false><<<grid, block, 0, st>>>(a, per_token);
  return cudaGetLastError();
}

template <bool INTER>
cudaError_t dispatch_rope(int D, bool mla, const RopeArgs& a, cudaStream_t st) {
  if (mla) {
    const unsigned per = kRopeThreads / 32;
    const unsigned grid = (a.tokens + per - 1) / per;
    if (a.slots)
      rope_mla_kernel<INTER, true><<<grid, kRopeThreads, 0, st>>>(a);
    else
      rope_mla_kernel<INTER, false><<<grid, kRopeThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  if (D == 64) return launch_rope_t<64, INTER>(a, st);
  if (D == 128) return launch_rope_t<128, INTER>(a, st);
  if (D == 256) return launch_rope_t<256, INTER>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(int D, bool mla, const RopeArgs& a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  return a.interleaved ? dispatch_rope<true>(D, mla, a, st) : dispatch_rope<false>(D, mla, a, st);
}

}  // namespace kvq
