// Per-head RMS norm and position rotation of queries and keys, and the append
// that applies them on the way into the paged cache (sm_103a).
//
// For one head x of D elements, all in fp32 from the bf16 input:
//   n_i = (x_i r) w_i,  r = RN(1 / sqrt(sum x^2 / D + eps))      (optional norm)
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
// pieces of two neighbouring lanes (rot is a multiple of 32).

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

constexpr int kRopeThreads = 256;
// From this many lanes (two thousand per SM) on, groups take kRowsEach rows.
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

__device__ __forceinline__ void load8f(const float* p, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// The eight angles of a lane's pairs, and the rotation of its 16 elements.
struct Angles {
  float c[8], s[8];
  // trow: the position's cosines, then (half further on) its sines
  __device__ __forceinline__ void load(const float* trow, int half, const Pieces& pc,
                                       bool interleaved) {
    // half-split order: the pairs' members lie at the same place in both
    // pieces; side by side: pairs 4 c0 .. 4 c0 + 3 in the first, 4 c1 .. in the
    // second
    const int i0 = interleaved ? 4 * pc.c0 : 8 * pc.c0, i1 = interleaved ? 4 * pc.c1 : i0 + 4;
    load4(trow + i0, c);
    load4(trow + i1, c + 4);
    load4(trow + half + i0, s);
    load4(trow + half + i1, s + 4);
  }
  static __device__ __forceinline__ void load4(const float* p, float* f) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  }
  __device__ __forceinline__ void turn(float& x, float& y, int i) const {
    const float a = x, b = y;
    x = __fmaf_rn(a, c[i], -__fmul_rn(b, s[i]));
    y = __fmaf_rn(b, c[i], __fmul_rn(a, s[i]));
  }
  __device__ __forceinline__ void apply(float (&f)[16], bool interleaved) const {
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(f[2 * i], f[2 * i + 1], i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(f[i], f[8 + i], i);
    }
  }
};

// 1 / rms of a row spread over LANES lanes (every lane of the warp calls it).
template <int LANES>
__device__ __forceinline__ float inv_rms(const float (&f)[16], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = __fmaf_rn(f[i], f[i], ss);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return __frsqrt_rn(ss * (1.0f / (LANES * 16)) + eps);   // the length is a power of two
}

__device__ __forceinline__ void apply_norm(float (&f)[16], float r, const float* w,
                                           const Pieces& pc) {
  float w0[8], w1[8];
  load8f(w + 8 * pc.c0, w0);
  load8f(w + 8 * pc.c1, w1);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = (f[i] * r) * w0[i];
    f[8 + i] = (f[8 + i] * r) * w1[i];
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float* f) {
  const uint32_t lo = f32x2_to_e4m3x2(f[0], f[1]) | (f32x2_to_e4m3x2(f[2], f[3]) << 16);
  const uint32_t hi = f32x2_to_e4m3x2(f[4], f[5]) | (f32x2_to_e4m3x2(f[6], f[7]) << 16);
  return make_uint2(lo, hi);
}

// E4M3(fl32(x / s)) of a lane's 16 elements (z = RN(1/s)).
__device__ __forceinline__ void store_e4m3(float (&f)[16], float s, float z, uint8_t* row,
                                           const Pieces& pc) {
  quotients_for_codes<16>(f, s, z, kE4m3Low);
  *reinterpret_cast<uint2*>(row + 8 * pc.c0) = pack_e4m3x8(f);
  *reinterpret_cast<uint2*>(row + 8 * pc.c1) = pack_e4m3x8(f + 8);
}

// One NVFP4 half block (8 elements; the neighbouring lane holds the other
// half): codes in a word, and the block's scale code.  Every lane of the warp
// calls it.
__device__ __forceinline__ uint32_t nvfp4_half(const float* x, float g, uint32_t& sc) {
  float bamax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) bamax = fmaxf(bamax, fabsf(x[i]));
  bamax = fmaxf(bamax, __shfl_xor_sync(0xffffffffu, bamax, 1));
  const float scf = __fdiv_rn(__fdiv_rn(bamax, 6.0f), g);
  sc = f32x2_to_e4m3x2(scf, 0.f) & 0xFFu;
  const float es = __fmul_rn(unpack_f16x2(e4m3x2_to_f16x2(sc)).x, g);
  if (es == 0.f) return 0u;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = x[i];
  quotients_for_codes<8>(f, es, __frcp_rn(es), kE2m1Low);
  return f32x8_to_e2m1x8(f);
}

// Both pieces of a lane as NVFP4 codes of cache row `row`; `ok` gates the stores.
template <int D>
__device__ __forceinline__ void store_nvfp4(float (&f)[16], float g, bool ok, uint8_t* codes,
                                            uint8_t* scales, long row, const Pieces& pc) {
  uint32_t s0, s1;
  const uint32_t w0 = nvfp4_half(f, g, s0), w1 = nvfp4_half(f + 8, g, s1);
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
// of range.
__device__ __forceinline__ long rope_page(const RopeArgs& a, const Token& k, bool report) {
  if (k.pos >= (long)a.max_pages * a.ps) return -1;
  const unsigned pos = (unsigned)k.pos, pi = pos / (unsigned)a.ps;
  const int page = __ldg(a.block_table + (size_t)k.b * a.max_pages + pi);
  if (page < 0 || page >= a.num_pages) {
    if (report) record_error(a.error_flag, 4);
    return -1;
  }
  return (long)page * a.Hkv * a.ps + (pos - pi * (unsigned)a.ps);
}

// FMT 0: bf16 rows out (kvq_norm_rope); otherwise K and V go to the cache.
// `per_token` lane groups of a block share a token (a power of two), and
// gridDim.y blocks: a group takes every (per_token gridDim.y)-th of its rows,
// the next row's loads going out before the present one's arithmetic.
template <int D, int FMT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int per_token) {
  // the append is an ordinary launch (it starts after all earlier work), the
  // other a programmatic one
  if constexpr (FMT == 0) griddep_wait();
  griddep_launch_dependents();
  constexpr int kLanes = D / 16, kGroups = kRopeThreads / kLanes;
  const int p = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const unsigned token = blockIdx.x * (unsigned)(kGroups / per_token) + group / per_token;
  const int H = a.q.heads + a.k.heads + a.v.heads;
  const int first = blockIdx.y * per_token + group % per_token, step = per_token * gridDim.y;
  const bool in = token < a.tokens;
  const Token tk = token_of(a, in ? token : 0, in && p == 0 && first == 0);
  const bool ok = in && tk.ok;

  // where row i of the token comes from
  auto source = [&](int i) -> const uint16_t* {
    const bool isq = i < a.q.heads, isv = i >= a.q.heads + a.k.heads;
    const RopeRows& src = isq ? a.q : isv ? a.v : a.k;
    const int h = i - (isq ? 0 : isv ? a.q.heads + a.k.heads : a.q.heads);
    return src.data + (long)token * src.token_stride + (long)h * src.head_stride;
  };
  const Pieces turned = pieces<D>(p, a.rot), plain = pieces<D>(p, 0);
  auto fetch = [&](int i, uint4& x0, uint4& x1) {
    x0 = x1 = make_uint4(0, 0, 0, 0);
    if (!ok || i >= H) return;
    const Pieces& pc = i < a.q.heads + a.k.heads ? turned : plain;
    const uint16_t* x = source(i);
    x0 = *reinterpret_cast<const uint4*>(x + 8 * pc.c0);
    x1 = *reinterpret_cast<const uint4*>(x + 8 * pc.c1);
  };
  uint4 x0, x1;
  fetch(first, x0, x1);
  Angles ang;
  if (turned.turn && ok)
    ang.load(a.cos_sin + tk.pos * a.rot, a.rot / 2, turned, a.interleaved != 0);
  // the page is the token's, whatever the head
  long page_row = -1;
  if constexpr (FMT != 0) page_row = ok ? rope_page(a, tk, p == 0 && first == 0) : -1;

#pragma unroll 1
  for (int i0 = 0; i0 < H; i0 += step) {   // the same rounds for every lane of the warp
    const int i = i0 + first;
    const bool row = ok && i < H;
    const bool isq = i < a.q.heads, isv = i >= a.q.heads + a.k.heads;
    const int h = i - (isq ? 0 : isv ? a.q.heads + a.k.heads : a.q.heads);
    const Pieces& pc = isv ? plain : turned;
    float f[16];
    bf16x8_to_f32(x0, f);
    bf16x8_to_f32(x1, f + 8);
    if (i0 + step < H) fetch(i + step, x0, x1);
    // every lane of the warp takes part in the norm's butterfly when any row
    // of the call has a norm
    const float* w = isq ? a.q_norm : isv ? nullptr : a.k_norm;
    if (a.q_norm || a.k_norm) {
      const float r = inv_rms<kLanes>(f, a.eps);
      if (w) apply_norm(f, r, w, pc);
    }
    if (turned.turn && !isv) ang.apply(f, a.interleaved != 0);

    if (isq || FMT == 0) {
      const RopeRows& dst = isq ? a.q_out : a.k_out;
      const long at = (long)token * dst.token_stride + (long)h * dst.head_stride;
      if (row) {
        if (isq && a.q_fp8) {
          const float s = a.q_hs ? __ldg(a.q_hs + h) : a.q_scale;
          const float z = a.q_hs ? __frcp_rn(s) : a.q_recip;
          store_e4m3(f, s, z, reinterpret_cast<uint8_t*>(dst.data) + at, pc);
        } else {
          *reinterpret_cast<uint4*>(dst.data + at + 8 * pc.c0) = pack_bf16x8(f);
          *reinterpret_cast<uint4*>(dst.data + at + 8 * pc.c1) = pack_bf16x8(f + 8);
        }
      }
    }
    if constexpr (FMT != 0) {
      const bool store = row && !isq && page_row >= 0;
      const long crow = page_row + (long)h * a.ps;
      const float* hs = isv ? a.v_hs : a.k_hs;
      const float s = (hs && store) ? __ldg(hs + h) : (isv ? a.v_scale : a.k_scale);
      if constexpr (FMT == kFmtFp8) {
        if (store) {
          const float z = hs ? __frcp_rn(s) : (isv ? a.v_recip : a.k_recip);
          store_e4m3(f, s, z, (isv ? a.v_codes : a.k_codes) + crow * D, pc);
        }
      } else {
        // lanes without a row stay for their neighbours' shuffles
        store_nvfp4<D>(f, s, store, isv ? a.v_codes : a.k_codes, isv ? a.v_bscale : a.k_bscale,
                       crow, pc);
      }
    }
  }
}

// MLA: one warp per token, the 512-wide latent (normed, then NVFP4) on all
// lanes, the 64 rope-key elements (rotated, bf16) on the first four.
__global__ void __launch_bounds__(kRopeThreads) rope_mla_kernel(const RopeArgs a) {
  griddep_launch_dependents();
  constexpr int D = 512, kRope = 64;
  const int lane = threadIdx.x & 31;
  const unsigned token = blockIdx.x * (unsigned)(kRopeThreads / 32) + threadIdx.x / 32;
  if (token >= a.tokens) return;   // the whole warp, as below
  const Token tk = token_of(a, token, lane == 0);
  const long crow = tk.ok ? rope_page(a, tk, lane == 0) : -1;
  if (crow < 0) return;

  const Pieces pc = pieces<D>(lane, 0);
  const uint16_t* x = a.k.data + (long)token * a.k.token_stride;
  float f[16];
  const uint4 x0 = *reinterpret_cast<const uint4*>(x + 8 * pc.c0);
  const uint4 x1 = *reinterpret_cast<const uint4*>(x + 8 * pc.c1);
  uint4 e0 = make_uint4(0, 0, 0, 0), e1 = e0;
  const Pieces pe = pieces<kRope>(lane & 3, a.rot);
  const uint16_t* xe = a.v.data + (long)token * a.v.token_stride;
  if (lane < kRope / 16) {
    e0 = *reinterpret_cast<const uint4*>(xe + 8 * pe.c0);
    e1 = *reinterpret_cast<const uint4*>(xe + 8 * pe.c1);
  }
  bf16x8_to_f32(x0, f);
  bf16x8_to_f32(x1, f + 8);
  if (a.k_norm) {
    const float r = inv_rms<32>(f, a.eps);
    apply_norm(f, r, a.k_norm, pc);
  }
  store_nvfp4<D>(f, a.k_scale, true, a.k_codes, a.k_bscale, crow, pc);
  if (lane < kRope / 16) {
    bf16x8_to_f32(e0, f);
    bf16x8_to_f32(e1, f + 8);
    if (pe.turn) {
      Angles ang;
      ang.load(a.cos_sin + tk.pos * a.rot, a.rot / 2, pe, a.interleaved != 0);
      ang.apply(f, a.interleaved != 0);
    }
    uint16_t* dst = a.k_pe + crow * kRope;
    *reinterpret_cast<uint4*>(dst + 8 * pe.c0) = pack_bf16x8(f);
    *reinterpret_cast<uint4*>(dst + 8 * pe.c1) = pack_bf16x8(f + 8);
  }
}

template <int D>
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
  if (a.fmt == 0) return launch_pdl(rope_kernel<D, 0>, grid, block, 0, st, a, per_token);
  if (a.fmt == kFmtFp8)
    rope_kernel<D, kFmtFp8><<<grid, block, 0, st>>>(a, per_token);
  else
    rope_kernel<D, kFmtNvfp4><<<grid, block, 0, st>>>(a, per_token);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int D, bool mla, const RopeArgs& a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  if (mla) {
    const unsigned per = kRopeThreads / 32;
    rope_mla_kernel<<<(a.tokens + per - 1) / per, kRopeThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  if (D == 64) return launch_rope_t<64>(a, st);
  if (D == 128) return launch_rope_t<128>(a, st);
  if (D == 256) return launch_rope_t<256>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
