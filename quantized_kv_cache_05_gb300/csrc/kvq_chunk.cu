// Causal attention of a packed ragged step over the quantized paged cache, on the
// 5th-generation tensor cores (sm_103a): prompt chunks, single tokens and idle requests
// in any mixture, with plain or differential heads.
//
// For one request and kv head the rows (new token i, query head g of the group) are a
// matrix Q [n G][D], row i G + g, whose row sees the keys 0 .. L - n + i:
//   S = sm_scale Q K^T,  P = exp(S - max) where the key is seen, else 0,  O = P V.
// A row tile is 256 such rows (two accumulators of 128; with 128 rows or fewer one, whose
// even and odd key tiles take turns), or 128 rows of differential heads, whose two maps
// take the two accumulators: S1 = Q1 K1^T and S2 = Q2 K2^T are products over half of the
// dims each, the values are shared.  The inner part -- the codes' way from TMA boxes to
// f16 operand tiles, the softmax of a row per thread with a lazily moving maximum, P in
// tensor memory -- is that of the shared prefix's kernel (kvq_shared.cu), where it is
// described.  What is different here:
//  * Shares.  Row tiles differ in their keys, so a grid over them leaves SMs idle, and a
//    few rows with many keys would use a few SMs.  All row tiles of all kv heads in one
//    line, each as long as its key tiles cost, are cut into equal shares, one per SM
//    (share_kernel); a CTA works on its share's pieces one after the other, the copies and
//    conversions of the next piece running on while the present one is written out.  A
//    row tile that a cut divides leaves partials (o normalized, lse) in the workspace, at
//    most two per CTA, which merge_kernel joins.
//  * Masks.  Only key tiles that reach past the first row's last key are masked, row by
//    row, by the thread that has the row.  Values of such a tile that are NaN (codes of a
//    NaN input) would reach rows that do not see them, as 0 NaN: there the tile's NaN rows
//    become zeros, and the rows that see one of them become NaN as a whole.
//  * Rounding.  P enters the products with V in two f16 parts (2^-21 of a weight, or 2^-31 of
//    the row's largest where that is more: f16's steps end at 2^-24, P is scaled by 2^7, and
//    each part may be off by half a step), as in the decode, so that as much is kept of a token's
//    weights whether its request brings one or many; where the caller asks for it, plain heads
//    have one (2^-11, against 2^-8 of the value that a bf16 output's rounding takes).  Differential heads always have two: their difference may
//    be small beside the two sums.  Sums and accumulators are fp32, long sums in chains
//    (kChainOne).
// Every wait is bounded; a timeout sets an error bit and the rows become NaN.
//
// What bounds it: 4096 rows x 32 heads (8 kv heads of 128, FP8) behind 12288 tokens take 1047
// us, 71% of the matrix rate with the second part's products (742 us), and 653 with one part
// of P (495, 76%); 2048 rows behind 6144 take 299 (FP8) and 326 (NVFP4), with one part 197 and
// 237.  With one part the tensor pipe is busy for 60% of the cycles and the schedulers issue in
// 45%: a key tile of two slots takes 1.9 us where its products need 1.05, each slot being a
// chain of scores, softmax and products, with some 200 cycles at every hand-over, and the codes
// of NVFP4 take the converting warps 1.74 us a tile.  With two parts it is some 2.8 us for 1.57:
// the softmax splits P and writes it twice.  Beside that a piece costs 7 us (queries
// 4, rows out 3), the shares' kernel 5 to 6, the single tokens 10 and more, the merge 7 to 19,
// one behind the other: of a step of a few hundred rows most of the 40 to 47 us.  Differential
// heads (four chunks of 1024, NVFP4: 441 us) spend 2.3 to 3 us on 128 rows' key tile, bound by
// the two parts of P.

#include <cfloat>
#include <climits>
#include <cstddef>
#include <type_traits>

#include "kvq_attn.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kTok = 128;                 // keys per tile, rows per accumulator
constexpr int kCol = kTok * 128;          // bytes of 64 f16 columns of 128 rows
// The issuing warps come first: an SM sub-core's scheduler prefers its oldest warp, and
// as the youngest the MMA warp took some 20 cycles an instruction, with every wait on the
// slots' critical path.
constexpr int kMmaWarp = 0, kTmaWarp = 1, kSoftWarp = 4, kConvWarp = 12;
constexpr int kSoftWarps = 8, kConvWarps = 4;   // softmax: four for each of the slots 0, 1
constexpr int kThreads = 512;             // four warpgroups: softmax x 2, convert, MMA and TMA
// Registers per thread of the warpgroups (the launch gives each thread 128, 512
// for the four): a softmax thread holds its row's 128 scores at once.
constexpr int kRegSoft = 176, kRegConv = 96, kRegIssue = 64;
static_assert(2 * kRegSoft + kRegConv + kRegIssue <= 4 * 128, "register pool of the launch");
constexpr float kPShift = 7.0f;           // log2 scale of P
// Units (key tiles of a slot) in a chain, whose products add up in TMEM.  The tensor cores
// cut off what does not fit an accumulator, always towards zero: 5e-8 of the sum for each
// product, 8 to a unit or 16 with two parts of P, so that with values of one sign 131072
// keys in one chain lost 1e-3 of a row.  A longer piece is a sum of
// chains, in fp32 rounded to nearest, kept in the workspace.  64 units with one part lose
// 2.5e-5 on average and up to 3.8e-5 (128: 5.6e-5 and 7.4e-5, in the same time); 32 with two
// parts 3.3e-5 (64: 6.5e-5; 4096 rows behind 12288 tokens: 3% less); 16 of
// differential heads 1.4e-5, nearly the same of both maps' sums (four chunks of 1024, NVFP4:
// 445 us against 429 in one chain); 4 of fp32 outputs 3.9e-6 (2048 rows behind 6144: 352 us
// against 299 with 32 units).  Powers of two: a unit's place in its chain is a
// mask.
constexpr int kChainOne = 64, kChainTwo = 32, kChainDiff = 16, kChainF32 = 4;
constexpr int kTmem = 512;                // S0 | S1 | O0 | O1, 128 columns each
constexpr int kRows = 2 * kTok;           // rows of a partial in the workspace

// Cost of a row tile, in twelfths of a key tile with both accumulators' rows (1.9 us): for
// each key tile 12, or with one accumulator's rows what its conversion takes (NVFP4: 1.74
// us; FP8: half of it, as two key tiles are on their way; with two parts of P 1.75 to 1.9 of
// 2.4 us), and kCostFixed for its queries and its output (7 us).  A share is at least
// kCostShare, a piece kMinPiece key tiles.
constexpr int kCostTwo = 12, kCostOneFp8 = 7, kCostOneNvfp4 = 11, kCostOneWide = 9;
constexpr int kCostFixed = 40, kCostShare = 64, kMinPiece = 3;

// ---------------------------------------------------------------------------
// Workspace: [head][cuts: grid + 1][requests: batch][lse: grid x 2 x kRows][o]
// ---------------------------------------------------------------------------
struct ChunkHead {
  int shares, active;     // CTAs with work; requests with new tokens
  int longest;            // single tokens up to this many keys are the decode's (kChunkLongest)
};
static_assert(offsetof(ChunkHead, longest) == kChunkLongest * sizeof(int), "read by the decode");
struct Cut {              // where a share begins: before key tile `kv` of a row tile
  int i, tile, h, kv;     // active request, row tile, kv head, key tile
  __device__ __forceinline__ bool tile_of(const Cut& o) const {
    return i == o.i && tile == o.tile && h == o.h;
  }
};
struct Request {
  int q0, n, L, b;        // first row, new tokens, keys, request
};

struct ChunkSpace {
  size_t cuts, requests, lse, o, bytes;
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
__host__ __device__ inline ChunkSpace chunk_space(int grid, int batch, int D) {
  ChunkSpace s;
  s.cuts = 256;
  s.requests = s.cuts + up256((size_t)(grid + 1) * sizeof(Cut));
  s.lse = s.requests + up256((size_t)batch * sizeof(Request));
  s.o = s.lse + up256((size_t)grid * 2 * kRows * sizeof(float));
  s.bytes = s.o + (size_t)grid * 2 * kRows * D * sizeof(float);
  return s;
}

// x / G for 0 <= x < 2^31, with the call's multiplier and shift (ChunkArgs): a division by
// a runtime number takes some twenty instructions, many times a piece.
__device__ __forceinline__ int over_g(const ChunkArgs& a, int x) {
  return (int)((__umulhi((unsigned)x, a.g_mul) + (unsigned)x) >> a.g_shift);
}

// Row tiles of a request with n new tokens, rt rows in each; the keys that the last
// row of tile j sees, and their tiles (at least one: rows that see nothing are written).
__device__ __forceinline__ int row_tiles(int n, int G, int rt) { return (n * G + rt - 1) / rt; }
__device__ __forceinline__ int keys_of(const Request& r, int G, int rt, int j) {
  const int e = min(r.n, ((j + 1) * rt - 1) / G + 1);
  return max(0, min(r.L, r.L - r.n + e));
}
__device__ __forceinline__ int key_tiles(int keys) { return max(1, (keys + kTok - 1) / kTok); }
__device__ __forceinline__ int tile_cost(const Request& r, int G, int rt, int one, int j) {
  const bool two = r.n * G - j * rt > kTok;   // (one: the cost with one accumulator's rows)
  return kCostFixed + (two ? kCostTwo : one) * key_tiles(keys_of(r, G, rt, j));
}

// ---------------------------------------------------------------------------
// Shares: one CTA lists the requests with new tokens, sums the costs of the row tiles
// (consecutive ones per thread) and finds the cuts, a thread per cut.
// ---------------------------------------------------------------------------
constexpr int kShareThreads = 256;
// The decode cuts every single token's keys into the same number of chunks, which the batch's
// capacity gives.  One whose chunks are longer than this, and than four times the mean over
// the decode's places (two CTAs on each SM), would keep a few SMs busy while the others, and
// the chunks' kernel, wait: it is cut into shares with the prompt chunks instead, where a key
// costs half as much again (batch 32 x 8 kv heads, one of 131072 keys and 31 of 1000: 148 us,
// by the decode alone 1107; two of 32768 and 30 idle ones 82 and 281.  With twice the mean 32
// of 1000 to 32000 keys take 413 us instead of 309).
constexpr int kLongChunk = 4096;

struct ShareSmem {
  long warp_a[kShareThreads / 32], warp_b[kShareThreads / 32];
  long start[kShareThreads];   // cost before each thread's tiles
};

__device__ __forceinline__ void scan2(long& a, long& b, long& total_a, long& total_b,
                                      ShareSmem& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sm.warp_a[warp] = a;
    sm.warp_b[warp] = b;
  }
  __syncthreads();
  long ta = 0, tb = 0;
  a -= a0;
  b -= b0;
#pragma unroll
  for (int i = 0; i < kShareThreads / 32; ++i) {
    if (i == warp) {
      a += ta;
      b += tb;
    }
    ta += sm.warp_a[i];
    tb += sm.warp_b[i];
  }
  total_a = ta;
  total_b = tb;
  __syncthreads();   // (the sums' places may be written again)
}

__global__ void __launch_bounds__(kShareThreads) share_kernel(const ChunkArgs a, int grid, int rt,
                                                              int one) {
  extern __shared__ int first[];   // row tiles before each active request
  __shared__ ShareSmem sm;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const ChunkSpace sp = chunk_space(grid, a.batch, a.D);
  if (a.counters)   // of the decode that takes the single tokens
    for (long i = tid; i < (long)a.batch * a.Hkv; i += kShareThreads) a.counters[i] = 0u;
  Cut* cuts = reinterpret_cast<Cut*>(a.workspace + sp.cuts);
  Request* requests = reinterpret_cast<Request*>(a.workspace + sp.requests);

  const int per = (a.batch + kShareThreads - 1) / kShareThreads;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  // ---- single tokens: those that the decode takes (kLongChunk)
  int longest = 0;
  if (a.counters) {
    long keys = 0, none = 0, unused;
    for (int b = b0; b < b1; ++b)
      if (min(max(a.q_offsets[b + 1], 0), a.num_tokens) -
              min(max(a.q_offsets[b], 0), a.num_tokens) == 1)
        keys += min(max(a.seq_lens[b], 0), a.max_kv_len);
    long all_keys;
    scan2(keys, none, all_keys, unused, sm);
    longest = (int)min(max((long)kLongChunk, 4 * all_keys * a.Hkv / (2 * grid)) * a.single_splits,
                       (long)INT_MAX);
    if (tid == 0) reinterpret_cast<ChunkHead*>(a.workspace)->longest = longest;
  }

  // ---- the active requests and their row tiles
  auto request = [&](int b) -> Request {
    Request r;
    r.q0 = min(max(a.q_offsets[b], 0), a.num_tokens);
    r.n = max(min(max(a.q_offsets[b + 1], 0), a.num_tokens) - r.q0, 0);
    const int len = a.seq_lens[b];
    r.L = min(max(len, 0), a.max_kv_len);
    if (a.counters && r.n == 1 && r.L <= longest) r.n = 0;   // the decode's
    if (r.L != len && r.n > 0) record_error(a.error_flag, 2);
    r.b = b;
    return r;
  };
  long active = 0, tiles = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request(b);
    active += r.n > 0;
    tiles += row_tiles(r.n, a.G, rt);
  }
  long all_active, T;
  scan2(active, tiles, all_active, T, sm);
  // more row tiles than all rows make: requests that share rows.  None is served (such
  // offsets could ask for any amount of work)
  const bool overlap = T > (long)a.num_tokens * a.G / rt + all_active;
  if (overlap) {
    T = 0;
    if (tid == 0) record_error(a.error_flag, 2);
  }
  const int A = overlap ? 0 : (int)all_active;
  for (int b = b0; b < b1 && !overlap; ++b) {
    const Request r = request(b);
    if (r.n == 0) continue;
    requests[active] = r;
    first[active] = (int)tiles;
    ++active;
    tiles += row_tiles(r.n, a.G, rt);
  }
  __syncthreads();

  // ---- the costs
  const long each = (T + kShareThreads - 1) / kShareThreads;
  const long t0 = min(tid * each, T), t1 = min(t0 + each, T);
  auto owner = [&](long t) -> int {   // the last request whose tiles begin at or before t
    int lo = 0, hi = A;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= t) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  long cost = 0, none = 0;
  if (t0 < t1) {
    int i = owner(t0);
    Request r = requests[i];
    for (long t = t0; t < t1; ++t) {
      if (i + 1 < A && t >= first[i + 1]) r = requests[++i];
      cost += tile_cost(r, a.G, rt, one, (int)(t - first[i]));
    }
  }
  long W, unused;   // of one kv head
  scan2(cost, none, W, unused, sm);
  sm.start[tid] = cost;
  __syncthreads();

  // ---- the cuts: share c begins at c / shares of the whole
  const long whole = W * a.Hkv;
  const int shares = (int)min((long)grid, (whole + kCostShare - 1) / kCostShare);
  if (tid == 0) *reinterpret_cast<ChunkHead*>(a.workspace) = ChunkHead{shares, A, longest};
  for (int c = tid; c <= shares && shares > 0; c += kShareThreads) {
    const long x = whole / shares * c + min((long)c, whole % shares);
    const int h = (int)(x / W);
    const long rem = x - h * W;
    Cut cut{0, 0, h, 0};
    if (rem > 0) {
      int lo = 0, hi = kShareThreads;   // the thread whose tiles hold it
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sm.start[mid] <= rem) lo = mid;
        else hi = mid;
      }
      // (threads without tiles begin where the last one with some ends)
      long t = min(lo * each, T - 1), at = sm.start[lo];
      int i = owner(t);
      Request r = requests[i];
      int tc = tile_cost(r, a.G, rt, one, (int)(t - first[i]));
      while (at + tc <= rem && t + 1 < T) {
        at += tc;
        ++t;
        if (i + 1 < A && t >= first[i + 1]) r = requests[++i];
        tc = tile_cost(r, a.G, rt, one, (int)(t - first[i]));
      }
      cut.i = i;
      cut.tile = (int)(t - first[i]);
      const int nk = key_tiles(keys_of(r, a.G, rt, cut.tile));
      int kv = (int)((rem - at) * nk / tc);
      // no pieces of less than kMinPiece key tiles
      if (kv < kMinPiece) {
        kv = 0;
      } else if (nk - kv < kMinPiece) {
        kv = 0;
        if (++cut.tile == row_tiles(r.n, a.G, rt)) {
          cut.tile = 0;
          if (++cut.i == A) {
            cut.i = 0;
            ++cut.h;
          }
        }
      }
      cut.kv = kv;
    }
    cuts[c] = cut;
  }
}

// ---------------------------------------------------------------------------
// Pieces of a share, in order.  Every warp walks them by itself.
// ---------------------------------------------------------------------------
struct Piece {
  Request r;
  int h, tile;
  int kv0, kv1, nk;       // key tiles of this piece, and of the row tile
  int keys;               // that the row tile's last row sees
};

struct Walk {
  Cut at, end;
  const Request* requests;
  int active, G, rt;
  __device__ __forceinline__ bool next(Piece& p) {
    if (at.tile_of(end) && at.kv >= end.kv) return false;
    p.r = requests[at.i];
    p.h = at.h;
    p.tile = at.tile;
    p.keys = keys_of(p.r, G, rt, at.tile);
    p.nk = key_tiles(p.keys);
    p.kv0 = at.kv;
    p.kv1 = at.tile_of(end) ? end.kv : p.nk;
    if (at.tile_of(end)) {
      at.kv = end.kv;
      return true;
    }
    at.kv = 0;
    if (++at.tile == row_tiles(p.r.n, G, rt)) {
      at.tile = 0;
      if (++at.i == active) {
        at.i = 0;
        ++at.h;
      }
    }
    return true;
  }
};

template <int FMT, int D>
struct ChunkGeom {
  using Gm = Geom<FMT, D>;
  static constexpr int kCols = D / 64;                  // 64-dim operand columns
  static constexpr int kTile = kCols * kCol;            // one f16 operand tile
  static constexpr int kRawCodes = kTok * Gm::kRow;
  static constexpr int kRaw = (kRawCodes + kTok * Gm::kSRow + 1023) / 1024 * 1024;
  static constexpr int kOffK = 2 * kTile;               // two Q tiles, then two K, two V
  static constexpr int kOffV = kOffK + 2 * kTile;
  static constexpr int kOffRaw = kOffV + 2 * kTile;
  // raw ring: as many K and V slots as fit, at most four
  static constexpr int kRoom = (229376 - kOffRaw) / (2 * kRaw);
  static constexpr int kSlots = kRoom < 4 ? kRoom : 4;
  static constexpr int kOffCtl = kOffRaw + 2 * kSlots * kRaw;
  static_assert(kSlots >= 1, "shared memory");
};

struct ChunkCtl {
  uint64_t raw_full[2][4], raw_empty[2][4];   // [K, V][slot]
  uint64_t op_full[2][2], op_empty[2][2];     // [K, V][operand tile]
  uint64_t s_full[2], p_full[2], o_full[2];   // per softmax slot
  uint64_t q_full, mma_done;
  uint32_t tmem;
  int abort_flag;
  uint32_t nan_rows[2][kTok / 32];            // of the V operand tiles (masked key tiles)
  // what the slots tell one another of their rows: with one accumulator's rows the score
  // scales (a[0]), then their states (a: maximum, b: sum); with differential heads the
  // factors of the sums (a) and the sums of squares of the halves (b)
  float a[2][kTok], b[2][kTok];
  // the softmax warps' places and pieces: their registers are for the scores
  Cut at[kSoftWarps], end;
  Piece piece[kSoftWarps];
};

// A row's 32 output elements in the output's type, 32 bytes at a time (each store touches a
// line for every row, and their number is what it costs: half of it with 32 bytes).
__device__ __forceinline__ void store_out32(void* out, int dtype, float scale, size_t at,
                                            const float (&v)[32]) {
  if (dtype == 0) {
    float* p = static_cast<float*>(out) + at;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v[8 * k + e];
      st_v8(p + 8 * k, x);
    }
    return;
  }
  if (dtype == 1) {
    float* p = reinterpret_cast<float*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[16 * k + 2 * e], v[16 * k + 2 * e + 1]);
        x[e] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h));
      }
      st_v8(p + 8 * k, x);
    }
    return;
  }
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float* q = v + 4 * e;
    x[e] = __uint_as_float(
        f32x2_to_e4m3x2(__fdiv_rn(q[0], scale), __fdiv_rn(q[1], scale)) |
        (f32x2_to_e4m3x2(__fdiv_rn(q[2], scale), __fdiv_rn(q[3], scale)) << 16));
  }
  st_v8(reinterpret_cast<float*>(static_cast<uint8_t*>(out) + at), x);
}

template <int FMT, int D, bool P2, bool DIFF>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const ChunkArgs a) {
  using Gm = Geom<FMT, D>;
  using Cg = ChunkGeom<FMT, D>;
  constexpr int kRt = DIFF ? kTok : kRows;   // rows of a row tile
  // units to a chain: plain heads with two parts of P know it by the output's type
  const int chain = DIFF ? kChainDiff : !P2 ? kChainOne : a.out_dtype == 0 ? kChainF32 : kChainTwo;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];   // the swizzle period
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(dyn_smem);
  ChunkCtl& sm = *reinterpret_cast<ChunkCtl*>(dyn_smem + Cg::kOffCtl);
  volatile int* abort_flag = &sm.abort_flag;

  if (warp == kTmaWarp && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < Cg::kSlots; ++k) {
        mbar_init(smem_u32(&sm.raw_full[i][k]), 1);
        mbar_init(smem_u32(&sm.raw_empty[i][k]), kConvWarps);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(smem_u32(&sm.op_full[i][k]), kConvWarps);
        mbar_init(smem_u32(&sm.op_empty[i][k]), 1);
      }
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), 4);
      mbar_init(smem_u32(&sm.o_full[i]), 1);
    }
    mbar_init(smem_u32(&sm.q_full), 8);
    mbar_init(smem_u32(&sm.mma_done), 1);
    sm.abort_flag = (base & 1023u) != 0;   // (never: the array is aligned)
    fence_barrier_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem)),
                 "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (warp == kMmaWarp && tmem != 0) *abort_flag = 1;   // (never: all of it is ours)
  // the shares' kernel has waited for everything earlier
  griddep_wait();
  griddep_launch_dependents();

  const ChunkSpace sp = chunk_space(gridDim.x, a.batch, D);
  const ChunkHead head = *reinterpret_cast<const ChunkHead*>(a.workspace);
  const Cut* cuts = reinterpret_cast<const Cut*>(a.workspace + sp.cuts);
  float* part_lse = reinterpret_cast<float*>(a.workspace + sp.lse);
  float* part_o = reinterpret_cast<float*>(a.workspace + sp.o);
  Walk walk;
  walk.requests = reinterpret_cast<const Request*>(a.workspace + sp.requests);
  walk.active = head.active;
  walk.G = a.G;
  walk.rt = kRt;
  walk.at = walk.end = Cut{0, 0, 0, 0};   // without a share: nothing
  if ((int)blockIdx.x < head.shares) {
    walk.at = cuts[blockIdx.x];
    walk.end = cuts[blockIdx.x + 1];
  }

  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
    if (wait_or_abort(smem_u32(&bar), parity, abort_flag)) return true;
    *abort_flag = 1;
    return false;
  };
  // Both accumulators have rows of their own (else the key tiles take turns)
  auto two_rows = [&](const Piece& p) -> bool {
    return DIFF || p.r.n * a.G - p.tile * kRt > kTok;
  };
  Piece p;

  if (warp < kSoftWarp) {
    regs_dec<kRegIssue>();
    if (warp == kTmaWarp) {
      // ================================================================= TMA
      int j = 0, issued[2] = {0, 0};   // key tiles of all pieces
      bool ok = true;
      while (ok && walk.next(p)) {
        const int32_t* table = a.block_table + (size_t)p.r.b * a.max_pages;
        for (int kv = p.kv0; kv < p.kv1 && ok; ++kv, ++j) {
          // lane i's cache row of box i (at most eight)
          const int valid = min(kTok, p.keys - kv * kTok);   // (<= 0: rows that see nothing)
          const int nb = valid > 0 ? (valid + a.box - 1) / a.box : 0;
          int row = 0;
          if (lane < nb) {
            const int tok = kv * kTok + lane * a.box, pidx = tok / a.ps;
            int page = __ldg(table + pidx);
            if (page < 0 || page >= a.num_pages) {
              record_error(a.error_flag, 4);
              page = 0;
            }
            row = (int)(((long)page * a.Hkv + p.h) * a.ps + (tok - pidx * a.ps));
          }
          const int rs = j % Cg::kSlots, turn = j / Cg::kSlots;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (turn > 0)
              ok = __all_sync(0xffffffffu, wait(sm.raw_empty[t][rs], (turn - 1) & 1));
            if (!ok) break;
            const uint32_t full = smem_u32(&sm.raw_full[t][rs]);
            const uint32_t dst = base + Cg::kOffRaw + (2 * rs + t) * Cg::kRaw;
            if (lane == 0) mbar_arrive_expect_tx(full, nb * a.box * (Gm::kRow + Gm::kSRow));
            __syncwarp();
            if (lane < nb) {
              tma_load_2d(dst + lane * a.box * Gm::kRow, t ? &tmV : &tmK, 0, row, full);
              if constexpr (FMT == kFmtNvfp4)
                bulk_load(dst + Cg::kRawCodes + lane * a.box * Gm::kSRow,
                          (t ? a.v_bscale : a.k_bscale) + (long)row * Gm::kSRow,
                          a.box * Gm::kSRow, full);
            }
            issued[t] = j + 1;
          }
        }
      }
      // no copy in flight at exit (bounded waits)
      if (lane == 0)
        for (int t = 0; t < 2; ++t)
          for (int i = max(0, issued[t] - Cg::kSlots); i < issued[t]; ++i)
            mbar_wait(smem_u32(&sm.raw_full[t][i % Cg::kSlots]), (i / Cg::kSlots) & 1);
    } else if (warp == kMmaWarp && elect_lane()) {
      // ================================================================= MMA
      // One thread, with as few instructions as there can be between a wait and the
      // products: beside the softmax warps each takes many cycles, and all of them are on
      // the slots' critical path.  Tensor memory starts at column 0 (all of it is this
      // CTA's).  A unit is a key tile in a slot: both slots take every tile, or turns.  In
      // its slot a unit's S follows the earlier one's P V, whose P's columns it needs, and
      // the two are issued together, so that the slots take turns on the tensor pipe, one in
      // its products while the other is in its softmax.  (A warp for each slot runs the
      // slots in step instead: 290 us against 208 for 2048 rows x 32 heads behind 6144
      // tokens.)
      constexpr uint32_t kIdS = idesc(0, 0, 0, kTok), kIdO = idesc(0, 0, 1, D);
      const uint64_t dq = sdesc(base, 16, 1024);
      const uint64_t dk = sdesc(base + Cg::kOffK, 16, 1024);
      const uint64_t dv = sdesc(base + Cg::kOffV, kCol, 1024);   // MN-major
      unsigned jk = 0, jv = 0;         // key tiles whose S, whose P V is issued
      unsigned taken[2] = {0, 0};      // units of each slot whose P has been taken
      // P V of key tile jv and S of key tile jk in a slot (either may be missing)
      auto step = [&](auto slot_c, bool product, bool score, bool two, bool acc) -> bool {
        constexpr int slot = decltype(slot_c)::value;
        // (a tile's V is converted before the next one's K)
        if (score) {
          if (!(two && slot == 1) && !wait(sm.op_full[0][jk & 1], (jk >> 1) & 1)) return false;
        } else if (!wait(sm.op_full[1][jv & 1], (jv >> 1) & 1)) {
          return false;
        }
        if (product) {
          const uint64_t v = dv + (jv & 1) * (unsigned)(Cg::kTile >> 4);
          constexpr uint32_t pc = slot * 128, o = 256 + slot * 128;
          if (!wait(sm.p_full[slot], taken[slot] & 1)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk) {
            const uint64_t vk = v + (kk * 2048 >> 4);
            if constexpr (P2) {   // high parts and residuals in alternating 16-column groups
              const uint32_t pk = pc + 32 * (kk >> 1) + 8 * (kk & 1);
              mma_ts(o, pk, vk, kIdO, kk > 0 || acc);
              mma_ts(o, pk + 16, vk, kIdO, true);
            } else {
              mma_ts(o, pc + 8 * kk, vk, kIdO, kk > 0 || acc);
            }
          }
          ++taken[slot];
        }
        if (score) {
          constexpr int kSteps = D / 16 / (DIFF ? 2 : 1);
          constexpr int k0 = DIFF ? slot * kSteps : 0;   // differential: the map's half of the dims
          const uint64_t k = dk + (jk & 1) * (unsigned)(Cg::kTile >> 4);
          const uint64_t q = dq + (two ? slot * Cg::kTile >> 4 : 0);
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const int kk = k0 + s;
            const uint64_t off = ((kk >> 2) * kCol + (kk & 3) * 32) >> 4;
            mma(slot * 128, q + off, k + off, kIdS, s > 0);
          }
          mma_commit(smem_u32(&sm.s_full[slot]));
        } else {                       // the slot's last of the piece
          mma_commit(smem_u32(&sm.o_full[slot]));
        }
        if (!two || slot == 1) {       // the tiles are free
          if (score) mma_commit(smem_u32(&sm.op_empty[0][jk++ & 1]));
          if (product) mma_commit(smem_u32(&sm.op_empty[1][jv++ & 1]));
        }
        return true;
      };
      using Zero = std::integral_constant<int, 0>;
      using One = std::integral_constant<int, 1>;
      unsigned pieces = 0;
      bool ok = true;
      while (ok && walk.next(p)) {
        const bool two = two_rows(p);
        const int nt = p.kv1 - p.kv0, units = two ? 2 * nt : nt;
        ok = wait(sm.q_full, pieces++ & 1);
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < units + 2 && ok; u += 2) {
          // (the first product of a chain overwrites)
          const bool acc = (((u >> 1) - 1) & (chain - 1)) != 0;
          if (u < units || u - 2 < units) ok = step(Zero{}, u >= 2, u < units, two, acc);
          if (ok && (u + 1 < units || (u >= 2 && u - 1 < units)))
            ok = step(One{}, u >= 2, u + 1 < units, two, acc);
        }
      }
      // every MMA has completed at exit (bounded wait)
      mma_commit(smem_u32(&sm.mma_done));
      mbar_wait(smem_u32(&sm.mma_done), 0);
    }
    __syncwarp();
  } else if (warp >= kConvWarp) {
    regs_dec<kRegConv>();
    // ============================================================= convert
    const int t = threadIdx.x - 32 * kConvWarp;
    const int px = t & 7, r = t;   // row r of the tile, row px of its 8-row atom
    int j = 0;
    bool ok = true;
    while (ok && walk.next(p)) {
      // keys that every row of the row tile sees
      const int all = p.r.L - p.r.n + over_g(a, p.tile * kRt) + 1;
      for (int kt = p.kv0; kt < p.kv1 && ok; ++kt, ++j) {
        const int rs = j % Cg::kSlots;
        const int nvalid = p.keys - kt * kTok;
        const bool masked = (kt + 1) * kTok > all;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t raw = base + Cg::kOffRaw + (2 * rs + kv) * Cg::kRaw;
          const uint32_t dst = base + (kv ? Cg::kOffV : Cg::kOffK) + (j & 1) * Cg::kTile +
                               (r >> 3) * 1024 + px * 128;
          ok = wait(sm.raw_full[kv][rs], (j / Cg::kSlots) & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          constexpr int kChunks = Gm::kRow / 16;
          uint4 v[kChunks];
          uint32_t sc[FMT == kFmtNvfp4 ? kChunks : 1];
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            v[c] = make_uint4(0u, 0u, 0u, 0u);
            if (r < nvalid) v[c] = lds128(raw + r * Gm::kRow + (Gm::swz(r, c) << 4));
          }
          if constexpr (FMT == kFmtNvfp4) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              sc[c] = r < nvalid ? lds16(raw + Cg::kRawCodes + r * Gm::kSRow + 2 * c) : 0u;
          }
          // the operand tile was last read by the MMAs of tile j - 2
          if (j >= 2) ok = wait(sm.op_empty[kv][j & 1], ((j >> 1) - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          if (kv == 1 && masked) {   // (warp-uniform) E4M3's NaN is 0x7F with either sign
            uint32_t bad = 0;
            if constexpr (FMT == kFmtFp8) {
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                bad |= __vcmpeq4(v[c].x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                       __vcmpeq4(v[c].y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                       __vcmpeq4(v[c].z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                       __vcmpeq4(v[c].w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            } else {
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                bad |= __vcmpeq4(sc[c] & 0x7F7Fu, 0x7F7F7F7Fu) & 0xFFFFu;
            }
            const uint32_t rows = __ballot_sync(0xffffffffu, bad != 0);
            if (lane == 0) sm.nan_rows[j & 1][r >> 5] = rows;
            if (bad) {
#pragma unroll
              for (int c = 0; c < kChunks; ++c) {
                v[c] = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (FMT == kFmtNvfp4) sc[c] = 0u;
              }
            }
          }
          if constexpr (FMT == kFmtFp8) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {   // 16 dims: two 16-byte pieces
              uint32_t o[8];
              e4m3x4_to_f16x2x2(v[c].x, o[0], o[1]);
              e4m3x4_to_f16x2x2(v[c].y, o[2], o[3]);
              e4m3x4_to_f16x2x2(v[c].z, o[4], o[5]);
              e4m3x4_to_f16x2x2(v[c].w, o[6], o[7]);
              const uint32_t row = dst + (c >> 2) * kCol;
              const int q = 2 * (c & 3);
              sts128(row + ((q ^ px) << 4), o[0], o[1], o[2], o[3]);
              sts128(row + (((q + 1) ^ px) << 4), o[4], o[5], o[6], o[7]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {   // 32 dims, two block scales
              const uint32_t s2 = e4m3x2_to_f16x2(sc[c]);
              const uint32_t s_lo = __byte_perm(s2, 0, 0x1010), s_hi = __byte_perm(s2, 0, 0x3232);
              const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
              const uint32_t row = dst + (c >> 1) * kCol;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t e0, e1, e2, e3;
                e2m1x8_to_f16x2x4(w[k], e0, e1, e2, e3);
                const uint32_t s = k < 2 ? s_lo : s_hi;
                const int q = 4 * (c & 1) + k;
                sts128(row + ((q ^ px) << 4), hmul2(e0, s), hmul2(e1, s), hmul2(e2, s),
                       hmul2(e3, s));
              }
            }
          }
          fence_proxy_async_shared();   // generic stores -> operands of the async MMAs
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&sm.op_full[kv][j & 1]));
            mbar_arrive(smem_u32(&sm.raw_empty[kv][rs]));
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
  } else {
    regs_inc<kRegSoft>();
    // ============================================================= softmax
    const int sw = warp - kSoftWarp, slot = sw >> 2, r = threadIdx.x & (kTok - 1);
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t sS = lane_addr + slot * 128, sO = lane_addr + 256 + slot * 128;
    unsigned j0 = 0;      // key tiles before the piece
    unsigned units = 0;   // of this slot, before the piece
    unsigned ends = 0;    // pieces before in which this slot had units
    bool ok = true;       // (after a timeout the pieces' barriers are still met)
    // The queries of a piece, into the slot's operand tile: their 16-byte pieces go straight
    // to the places that their f16 values take, FP8 codes at every other one (they widen to
    // two); consecutive lanes copy consecutive pieces, and rows past the last are zeros.
    // Plain heads' next piece's are on their way while rows are written (4096 rows behind 12288
    // tokens: 1047 us against 1105, with one part of P 660 against 676; with differential heads
    // this loses, 444 against 424 for four chunks of 1024: the kernel's code is larger).
    constexpr int kHalf = DIFF ? 2 : 1;                             // of the dims in an operand
    const int dp0 = DIFF ? slot * (D / 16) : 0;                     // its first piece (8 dims each)
    auto q_place = [&](bool two, int trow, int piece) -> uint32_t {
      return base + (two ? slot * Cg::kTile : 0) + (piece >> 3) * kCol + (trow >> 3) * 1024 +
             (trow & 7) * 128 + (((piece ^ trow) & 7) << 4);
    };
    auto fetch_q = [&](const Piece& p) {
      const bool two = two_rows(p);
      if (!two && slot == 1) return;
      const int R = p.r.n * a.G;
      const int lp = (a.q_fp8 ? D / 16 : D / 8) / kHalf;            // pieces of a row
      const int c = lane & (lp - 1), per = 32 / lp, trow = 32 * (warp & 3) + lane / lp;
      const int first = p.tile * kRt + (two && !DIFF ? slot * kTok : 0) + trow;
      // row first + k per: token qt, head qg of the group, without a division each
      int qt = over_g(a, first), qg = first - qt * a.G;
      const int dt = over_g(a, per), dg = per - dt * a.G;
      const long row_bytes = a.q_fp8 ? D : 2 * D;
      const uint8_t* q0 = static_cast<const uint8_t*>(a.q) +
                          ((long)p.r.q0 * a.Hq + (long)p.h * a.G) * row_bytes + 16 * c +
                          (DIFF ? slot * (row_bytes / 2) : 0);
#pragma unroll 4
      for (int k = 0; k < lp; ++k) {
        const bool in = first + k * per < R;
        const uint8_t* src = in ? q0 + ((long)qt * a.Hq + qg) * row_bytes : q0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(
                         q_place(two, trow + k * per, dp0 + (a.q_fp8 ? 2 * c : c))),
                     "l"(src), "r"(in ? 16 : 0)
                     : "memory");
        qt += dt;
        qg += dg;
        if (qg >= a.G) {
          qg -= a.G;
          ++qt;
        }
      }
    };
    bool fetched = false;   // this piece's queries are on their way
    auto fetch_next = [&] {
      Walk w = walk;
      Piece next;
      w.at = sm.at[sw];
      w.end = sm.end;
      fetched = w.next(next);
      if (fetched) fetch_q(next);
    };
    if (lane == 0) sm.at[sw] = walk.at;
    if (threadIdx.x == 32 * kSoftWarp) sm.end = walk.end;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    while (true) {
      {
        Walk w = walk;
        w.at = sm.at[sw];
        w.end = sm.end;
        if (!w.next(p)) break;
        __syncwarp();
        if (lane == 0) {
          sm.at[sw] = w.at;
          sm.piece[sw] = p;
        }
        __syncwarp();
      }
      const bool two = two_rows(p);
      const int nt = p.kv1 - p.kv0;
      const int R = p.r.n * a.G;                                    // the request's rows
      const int row = p.tile * kRt + (two && !DIFF ? slot * kTok : 0) + r;
      const bool live = row < R;
      const int ti = live ? over_g(a, row) : 0, g = live ? row - ti * a.G : 0;
      const int hq = p.h * a.G + g;
      const int seen = live ? p.r.L - p.r.n + ti + 1 : INT_MAX;    // keys of this row

      // ---- the rows' queries, in their operand tile
      auto q_at = [&](int trow, int piece) -> uint32_t { return q_place(two, trow, piece); };
      // Score scale, log2 domain: positive, so that the row's largest score is that of
      // its largest product and the -inf of a key that is not seen stays one.  A scale
      // below zero (a query head's) turns the query's sign instead; one of zero, also by
      // underflow, counts as the smallest normal number.
      float qsc = 0.f;
      if (two || slot == 0) {
        if (!fetched) fetch_q(p);
        const float k_log2 = (a.k_hs ? a.sm_scale * __ldg(a.k_hs + p.h) : a.sm_scale * a.k_scale) *
                             1.4426950408889634f;
        uint32_t flip = 0u;   // sign bits of a pair, where the query's sign turns
        auto settle_scale = [&](float s) {
          if (s < 0.f) flip = 0x80008000u;
          qsc = s == 0.f ? FLT_MIN : fabsf(s);   // (NaN stays)
        };
        if (a.q_fp8) settle_scale(k_log2 * (a.q_hs ? __ldg(a.q_hs + hq) : a.q_scale));
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();   // the warp's rows are here
        constexpr int kQ = D / 8 / kHalf;   // f16 pieces of the row
        uint4 v[kQ];                         // (all loads at once; the scores are not here yet)
#pragma unroll
        for (int c = 0; c < kQ; ++c)
          if (!(a.q_fp8 && (c & 1))) v[c] = lds128(q_at(r, dp0 + c));
        if (a.q_fp8) {
#pragma unroll
          for (int c = 0; c < kQ; c += 2) {   // 16 codes as two f16 pieces
            uint32_t o[8];
            e4m3x4_to_f16x2x2(v[c].x, o[0], o[1]);
            e4m3x4_to_f16x2x2(v[c].y, o[2], o[3]);
            e4m3x4_to_f16x2x2(v[c].z, o[4], o[5]);
            e4m3x4_to_f16x2x2(v[c].w, o[6], o[7]);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] ^= flip;
            sts128(q_at(r, dp0 + c), o[0], o[1], o[2], o[3]);
            sts128(q_at(r, dp0 + c + 1), o[4], o[5], o[6], o[7]);
          }
        } else {
          // prescaled by a power of two, so that the f16 values are exact
          uint32_t m2 = 0;   // the largest magnitudes of the even and odd elements
#pragma unroll
          for (int c = 0; c < kQ; ++c)
            m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu),
                                       __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu)));
          const int e = q_prescale_exp(max(m2 & 0xFFFFu, m2 >> 16));
          settle_scale(scale_pow2(k_log2, -e));
          const float f = exp2i(e);
#pragma unroll
          for (int c = 0; c < kQ; ++c) {
            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = pack_f16x2(__uint_as_float(w[k] << 16) * f,
                                __uint_as_float(w[k] & 0xFFFF0000u) * f) ^ flip;
            sts128(q_at(r, dp0 + c), o[0], o[1], o[2], o[3]);
          }
        }
        fence_proxy_async_shared();
        if (!two) sm.a[0][r] = qsc;
      }
      if (!two) {   // slot 1 has the same rows
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (slot == 1) qsc = sm.a[0][r];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.q_full));

      fetched = false;

      // ---- the slot's units
      const int cnt = two ? nt : (nt + 1 - slot) / 2;
      float m = -INFINITY, l = 0.f;   // reference max (log2), sum of 2^(x - m + 7)
      bool poison = false;            // sees a token whose values are NaN
      // keys from the piece's first on that this row sees, and that every row does
      const int mine = seen - p.kv0 * kTok;
      const int every = p.r.L - p.r.n + over_g(a, p.tile * kRt) + 1 - p.kv0 * kTok;
      asm volatile("" ::: "memory");   // (what follows reads the piece from shared memory)
      float held = -INFINITY;         // the reference of what the chains before have left
      // its place in the workspace, the share's last partial's: [8-dim column][row][8]
      auto chain_at = [&](int col8) -> float* {
        return part_o + (size_t)(2 * blockIdx.x + 1) * kRows * D + (slot * kTok + r) * 8 +
               (size_t)col8 * kRows * 8;
      };
      int i = 0;
#pragma unroll 1
      while (true) {   // a chain at a time
        for (const int end = min(i + chain, cnt); i < end && ok; ++i) {
          const int jj = two ? i : 2 * i + slot;         // key tile of the piece
          const int nvalid = mine - jj * kTok;           // keys of this tile that the row sees
          ok = __all_sync(0xffffffffu, wait(sm.s_full[slot], (units + i) & 1));
          if (!ok) break;
          tc_fence_after();
          uint32_t s[4][32];   // the row's scores
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(sS + 32 * c, s[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld32(s[c]);
          if ((jj + 1) * kTok > every) {   // some row does not see all of it
            if (__any_sync(0xffffffffu, nvalid < kTok)) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (32 * c + k >= nvalid) s[c][k] = 0xFF800000u;   // -inf
            }
            // the V operand tile of the same number: converted, with its NaN rows listed
            const unsigned j = j0 + jj;
            ok = __all_sync(0xffffffffu, wait(sm.op_full[1][j & 1], (j >> 1) & 1));
            if (!ok) break;
#pragma unroll
            for (int w = 0; w < kTok / 32; ++w) {
              const int upto = nvalid - 32 * w;   // of this word's rows, those that are seen
              const uint32_t seen_rows =
                  upto >= 32 ? 0xffffffffu : upto <= 0 ? 0u : (1u << upto) - 1u;
              poison |= (*(volatile uint32_t*)&sm.nan_rows[j & 1][w] & seen_rows) != 0u;
            }
          }
          float mx4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx4[c] = __uint_as_float(s[c][0]);
#pragma unroll
            for (int k = 1; k < 31; k += 2)
              mx4[c] = max3(mx4[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
            mx4[c] = fmaxf(mx4[c], __uint_as_float(s[c][31]));
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * qsc;
          const bool move = mx > m + kLazyMax;   // also the first finite tile
          if (__any_sync(0xffffffffu, move)) {
            const float alpha = move ? ex2(m - mx) : 1.f;
            m = move ? mx : m;
            l *= alpha;
            // O of the slot's earlier units (complete: this unit's S was committed
            // after them)
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(sO + 16 * c, o);
                tmem_wait_ld16(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st16(sO + 16 * c, o);
              }
            }
          }
          const float ref = (m == -INFINITY ? 0.f : m) - kPShift;
          const uint64_t q2 = pack2(qsc, qsc), r2 = pack2(-ref, -ref);
          uint64_t sum2 = 0ull;   // two zeros
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 x = unpack2(fma2(
                  pack2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), q2, r2));
              const float p0 = ex2(x.x), p1 = ex2(x.y);
              sum2 = add2(sum2, pack2(p0, p1));
              if constexpr (P2) {   // the leading 11 bits, and what is left
                const float h0 = __uint_as_float(__float_as_uint(p0) & 0xFFFFE000u);
                const float h1 = __uint_as_float(__float_as_uint(p1) & 0xFFFFE000u);
                hi[k] = pack_f16x2(h0, h1);
                const float2 r = unpack2(fma2(pack2(h0, h1), pack2(-1.f, -1.f), pack2(p0, p1)));
                lo[k] = pack_f16x2(r.x, r.y);
              } else {
                hi[k] = pack_f16x2(p0, p1);
              }
            }
            tmem_st16(sS + (P2 ? 32 * c : 16 * c), hi);
            if constexpr (P2) tmem_st16(sS + 32 * c + 16, lo);
          }
          // P is written (and O rescaled): its products may go.  (Handed over in halves, each
          // with a wait of its own: 722 us against 685 for 4096 rows x 32 heads behind 12288
          // tokens.)
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[slot]));
          const float2 sum = unpack2(sum2);
          l += sum.x + sum.y;
        }
        // The chain's products are complete with the next unit's scores, whose product
        // overwrites O.
        if (i >= cnt || !ok) break;
        ok = __all_sync(0xffffffffu, wait(sm.s_full[slot], (units + i) & 1));
        if (!ok) break;
        tc_fence_after();
        const float f = held == m ? 1.f : ex2(held - m);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(sO + 16 * c, o);
          tmem_wait_ld16(o);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[8] = {};
            if (i > chain) ld_v8(chain_at(2 * c + h), x);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = x[k] * f + __uint_as_float(o[8 * h + k]);
            st_v8(chain_at(2 * c + h), x);
          }
        }
        held = m;
      }
      if (poison) l = NAN;
      j0 += nt;
      units += cnt;
      __syncwarp();
      p = *const_cast<const Piece*>(&sm.piece[sw]);

      // ---- the rows' results
      asm volatile("" ::: "memory");
      // f[s] is the factor of slot s's accumulator, lse the row's.  Joined (one
      // accumulator's rows, or differential heads written whole): each slot does half of
      // the dims of both accumulators.
      const bool whole = p.kv0 == 0 && p.kv1 == p.nk;
      const bool join = !two || (DIFF && whole);
      const float out_mult = a.v_hs ? __ldg(a.v_hs + p.h) : a.v_scale;
      float lse = -INFINITY;
      // the factors of the sums with (maximum, sum) (m0, l0) and (m1, l1) in one row
      auto factors = [&](float m0, float l0, float m1, float l1, float& f0, float& f1) {
        const float M = fmaxf(m0, m1);
        const float e0 = m0 == -INFINITY ? 0.f : ex2(m0 - M);
        const float e1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
        // l0, l1 may be NaN (a NaN or infinite score): it passes through
        const float L = e0 * l0 + e1 * l1;
        f0 = f1 = 0.f;
        if (M != -INFINITY && L != 0.f) {
          f0 = e0 / L * out_mult;
          f1 = e1 / L * out_mult;
          lse = (M - kPShift + log2f(L)) * kLn2;
        } else if (!(l0 == 0.f && l1 == 0.f)) {
          f0 = f1 = NAN;
          lse = NAN;
        }
      };
      float own = 0.f, unused;
      if (two) factors(m, l, -INFINITY, 0.f, own, unused);
      if (DIFF && join && slot == 1) own *= -__ldg(a.diff_lambda + hq);
      if (join) {
        sm.a[slot][r] = two ? own : m;
        if (!two) sm.b[slot][r] = l;
      }
      if (cnt > 0) ok = ok && wait(sm.o_full[slot], ends++ & 1);
      if (cnt > chain) {   // the chains together
        tc_fence_after();
        const float f = held == m ? 1.f : ex2(held - m);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(sO + 16 * c, o);
          tmem_wait_ld16(o);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[8];
            ld_v8(chain_at(2 * c + h), x);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o[8 * h + k] = __float_as_uint(__uint_as_float(o[8 * h + k]) + x[k] * f);
          }
          tmem_st16(sO + 16 * c, o);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      if (join) asm volatile("bar.sync 1, 256;" ::: "memory");   // both accumulators are done
      const bool bad = __any_sync(0xffffffffu, !ok || *abort_flag != 0);
      ok = !bad;
      tc_fence_after();
      if constexpr (!DIFF) fetch_next();   // (before the rows are written)
      float f[2];
      if (!two) {
        factors(sm.a[0][r], sm.b[0][r], sm.a[1][r], sm.b[1][r], f[0], f[1]);
      } else {
        f[0] = join ? sm.a[0][r] : own;
        f[1] = join ? sm.a[1][r] : own;
      }
      // 32 dims of the row: both accumulators', or this slot's
      const bool use0 = join || slot == 0, use1 = join ? two || nt > 1 : slot == 1;
      auto take = [&](int c, float (&o)[32]) {
        uint32_t s[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0.f;
        if (use0) {
          tmem_ld32(lane_addr + 256 + 32 * c, s);
          tmem_wait_ld32(s);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(s[k]) * f[0];
        }
        if (use1) {
          tmem_ld32(lane_addr + 256 + 128 + 32 * c, s);
          tmem_wait_ld32(s);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] += __uint_as_float(s[k]) * f[1];
        }
        if (bad) {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = NAN;
        }
      };
      const int nc = join ? D / 64 : D / 32, c0 = join ? slot * nc : 0;   // its 32-dim columns
      const size_t out_row = ((size_t)(p.r.q0 + ti) * a.Hq + hq) * D;
      if (DIFF && whole) {
        float y[D / 64][32];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          take(c0 + c, y[c]);
#pragma unroll
          for (int k = 0; k < 32; ++k) ss += y[c][k] * y[c][k];
        }
        float rr = a.diff_gain;
        if (a.diff_norm) {   // (uniform)
          sm.b[slot][r] = ss;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          rr *= inv_rms_of((sm.b[0][r] + sm.b[1][r]) * (1.f / D) + a.diff_eps);
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
            if (a.diff_norm)
              w = __ldg(reinterpret_cast<const float4*>(a.diff_norm + 32 * (c0 + c) + k));
            y[c][k] *= rr * w.x;
            y[c][k + 1] *= rr * w.y;
            y[c][k + 2] *= rr * w.z;
            y[c][k + 3] *= rr * w.w;
          }
          if (live) store_out32(a.out, a.out_dtype, a.out_scale, out_row + 32 * (c0 + c), y[c]);
        }
      } else if (whole) {
#pragma unroll 1
        for (int c = c0; c < c0 + nc; ++c) {
          float o[32];
          take(c, o);
          if (live) store_out32(a.out, a.out_dtype, a.out_scale, out_row + 32 * c, o);
        }
      } else {
        // a partial: where the piece begins the row tile it is the share's last
        const int at = 2 * blockIdx.x + (p.kv0 == 0 ? 1 : 0);
        const int prow = (two ? slot * kTok : 0) + r;
        if (live && (two || slot == 0)) part_lse[(size_t)at * kRows + prow] = bad ? NAN : lse;
        // [8-dim column][row][8]: neighbouring lanes' rows lie side by side
        float* po = part_o + (size_t)at * kRows * D + prow * 8;
#pragma unroll 1
        for (int c = c0; c < c0 + nc; ++c) {
          float o[32];
          take(c, o);
          if (live) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = o[8 * k + e];
              st_v8(po + (size_t)(4 * c + k) * kRows * 8, v);
            }
          }
        }
      }
      // the other slot's next unit overwrites what this one has read of its accumulator
      // and its state
      if (join) {
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tc_fence_after();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) record_error(a.error_flag, 1);
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem)
                 : "memory");
  }
}

// The larger of two numbers; NaN where either is.
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------------------
// Merge of the row tiles that cuts divide (M = max lse, w_j = e^(lse_j - M), O = sum w_j
// o_j / sum w_j, 0 when all are empty), a warp for a few rows at once.  Blocks (x, y): the
// tile that begins in share y and goes on in the next.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 8, kMergeRows = 4;   // rows of a warp: their loads overlap

template <int D, bool DIFF>
__global__ void __launch_bounds__(32 * kMergeWarps)
    merge_kernel(const ChunkArgs a, int grid) {
  constexpr int kRt = DIFF ? kTok : kRows;
  constexpr int kMaps = DIFF ? 2 : 1;
  constexpr int NR = kMergeRows / kMaps;   // rows in one go, with their maps
  constexpr int kPer = D / 32;             // dims per lane
  using Vec = std::conditional_t<kPer == 4, float4, float2>;
  griddep_wait();
  griddep_launch_dependents();
  const ChunkSpace sp = chunk_space(grid, a.batch, D);
  const ChunkHead head = *reinterpret_cast<const ChunkHead*>(a.workspace);
  const Cut* cuts = reinterpret_cast<const Cut*>(a.workspace + sp.cuts);
  const int share = blockIdx.y;
  if (share >= head.shares) return;
  const Cut begin = cuts[share], cut = cuts[share + 1];
  // a cut inside a row tile that begins in this share
  if (cut.kv == 0 || (begin.tile_of(cut) && begin.kv > 0)) return;
  const Request q = reinterpret_cast<const Request*>(a.workspace + sp.requests)[cut.i];
  const int lane = threadIdx.x & 31;
  const int rows = min(kRt, q.n * a.G - cut.tile * kRt);   // of the tile
  const float* part_lse = reinterpret_cast<const float*>(a.workspace + sp.lse);
  const float* part_o = reinterpret_cast<const float*>(a.workspace + sp.o) +
                        (size_t)(lane * kPer / 8) * kRows * 8 + lane * kPer % 8;
  // pieces: this share's last, then the first ones of the following shares up to the one
  // that ends the row tile (shares without any key tile have none)
  int last = share + 1;
  while (last < head.shares && cuts[last + 1].tile_of(cut) && cuts[last + 1].kv > 0) ++last;
  const int pieces = last - share + 1;
  auto slot_of = [&](int j) -> size_t { return j == 0 ? 2 * share + 1 : 2 * (share + j); };
  auto empty = [&](int j) -> bool {
    return j > 0 && cuts[share + j].tile_of(cuts[share + j + 1]) &&
           cuts[share + j].kv == cuts[share + j + 1].kv;
  };

  const int warps = gridDim.x * kMergeWarps;
  for (int r0 = NR * (blockIdx.x * kMergeWarps + (threadIdx.x >> 5)); r0 < rows; r0 += NR * warps) {
    // row i of the partials: rows r0 .., the maps of one after the other
    auto prow = [&](int i) -> int { return min(r0 + i / kMaps, rows - 1) + (i % kMaps) * kTok; };
    float M[kMergeRows], sum[kMergeRows], o[kMergeRows][kPer];
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i) {
      M[i] = -INFINITY;
      sum[i] = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[i][e] = 0.f;
    }
    for (int j = lane; j < pieces; j += 32) {
      const bool none = empty(j);
#pragma unroll
      for (int i = 0; i < kMergeRows; ++i)
        if (!none) M[i] = nan_max(M[i], part_lse[slot_of(j) * kRows + prow(i)]);
    }
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i)
#pragma unroll
      for (int k = 16; k > 0; k >>= 1)
        M[i] = nan_max(M[i], __shfl_xor_sync(0xffffffffu, M[i], k));
    for (int j0 = 0; j0 < pieces; j0 += 32) {
      const bool some = j0 + lane < pieces && !empty(j0 + lane);
      float w[kMergeRows];
#pragma unroll
      for (int i = 0; i < kMergeRows; ++i) {
        const float x = some ? part_lse[slot_of(j0 + lane) * kRows + prow(i)] : -INFINITY;
        w[i] = x == -INFINITY ? 0.f : expf(x - M[i]);
        sum[i] += w[i];
      }
      const int n = min(32, pieces - j0);
#pragma unroll 2
      for (int j = 0; j < n; ++j) {
        // (a share without a piece leaves nothing to read)
        const bool here = __shfl_sync(0xffffffffu, (int)some, j) != 0;
        Vec v[kMergeRows];
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i)
          if (here)
            v[i] = *reinterpret_cast<const Vec*>(part_o + slot_of(j0 + j) * kRows * D +
                                                 (size_t)prow(i) * 8);
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i) {
          const float wj = __shfl_sync(0xffffffffu, w[i], j);
          const float* f = reinterpret_cast<const float*>(&v[i]);
          if (here && wj != 0.f) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[i][e] += wj * f[e];
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i) {
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], k);
      const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[i][e] *= inv;
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = cut.tile * kRt + r0 + n;
      if (r0 + n >= rows) break;
      float* y = o[kMaps * n];
      const int ti = over_g(a, row), hq = cut.h * a.G + (row - ti * a.G);
      if constexpr (DIFF) {
        const float lam = __ldg(a.diff_lambda + hq);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          y[e] -= lam * o[kMaps * n + 1][e];
          ss += y[e] * y[e];
        }
        float rr = a.diff_gain;
        if (a.diff_norm) {
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
          rr *= inv_rms_of(ss * (1.f / D) + a.diff_eps);
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          y[e] *= rr * (a.diff_norm ? __ldg(a.diff_norm + lane * kPer + e) : 1.f);
      }
      const size_t at = ((size_t)(q.q0 + ti) * a.Hq + hq) * D + lane * kPer;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (a.out_dtype == 0) store_out_t<0>(a.out, a.out_scale, at + e, y[e]);
        else if (a.out_dtype == 1) store_out_t<1>(a.out, a.out_scale, at + e, y[e]);
        else store_out_t<2>(a.out, a.out_scale, at + e, y[e]);
      }
    }
  }
}

template <int FMT, int D, bool P2, bool DIFF>
cudaError_t launch_t(const TensorMaps& m, const ChunkArgs& a, int grid, cudaStream_t st) {
  using Cg = ChunkGeom<FMT, D>;
  constexpr size_t smem = Cg::kOffCtl + sizeof(ChunkCtl);
  static_assert(smem <= 232448, "shared memory of one CTA");
  auto kern = chunk_kernel<FMT, D, P2, DIFF>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, m.k16, m.v16, a);
  if (e != cudaSuccess) return e;
  // (eight blocks for a divided tile: all of them run at once)
  return launch_pdl(merge_kernel<D, DIFF>, dim3(8, grid), dim3(32 * kMergeWarps), 0, st, a, grid);
}

template <int FMT, int D>
cudaError_t by_kind(const TensorMaps& m, const ChunkArgs& a, int grid, cudaStream_t st) {
  if (a.diff_lambda) return launch_t<FMT, D, true, true>(m, a, grid, st);
  if (a.wide_p) return launch_t<FMT, D, true, false>(m, a, grid, st);
  return launch_t<FMT, D, false, false>(m, a, grid, st);
}

}  // namespace

cudaError_t launch_shares(int fmt, const ChunkArgs& a, int grid, cudaStream_t st) {
  constexpr size_t kMost = (size_t)kMaxPlanBatch * sizeof(int);
  static_assert(kMost + sizeof(ShareSmem) <= 232448, "shared memory of one CTA");
  cudaError_t e =
      cudaFuncSetAttribute(share_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
  if (e != cudaSuccess) return e;
  const bool diff = a.diff_lambda != nullptr;
  const int one = diff                ? kCostTwo
                  : a.wide_p          ? kCostOneWide
                  : fmt == kFmtFp8    ? kCostOneFp8
                                      : kCostOneNvfp4;
  return launch_pdl(share_kernel, dim3(1), dim3(kShareThreads), (size_t)a.batch * sizeof(int), st,
                    a, grid, diff ? kTok : kRows, one);
}

size_t chunk_workspace_bytes(int grid, int batch, int D) { return chunk_space(grid, batch, D).bytes; }

cudaError_t launch_chunk(int fmt, int D, const TensorMaps& m, const ChunkArgs& a, int grid,
                         cudaStream_t st) {
  if (fmt == kFmtFp8 && D == 128) return by_kind<kFmtFp8, 128>(m, a, grid, st);
  if (fmt == kFmtFp8 && D == 64) return by_kind<kFmtFp8, 64>(m, a, grid, st);
  if (fmt == kFmtNvfp4 && D == 128) return by_kind<kFmtNvfp4, 128>(m, a, grid, st);
  if (fmt == kFmtNvfp4 && D == 64) return by_kind<kFmtNvfp4, 64>(m, a, grid, st);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
