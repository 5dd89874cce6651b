// Attention of a whole batch's query rows over a prefix that all requests
// share, on the 5th-generation tensor cores (sm_103a).
//
// All B requests hold the same first tokens, in the same pages.  For one kv
// head the rows q[b][g] of its B x G query heads are then one matrix Q [R][D],
// and the prefix's part of the split-KV decode is one attention
//   S = sm_scale Q K^T,  P = exp(S - max),  O = P V
// that reads K and V once for every 256 rows instead of once per request.  The
// kernel writes it as split partials (o normalized, lse) of the shape that the
// split-KV decode merges; the decode kernel does the requests' own tokens and
// the merge.  Rows of requests shorter than the prefix take no part (their
// partial is empty; the decode kernel reads all their tokens).
//
// One CTA per SM runs one split for MT x 128 rows, in tiles of 128 tokens:
//  * a TMA warp brings the tile's codes (boxes of whole 16- to 128-token page
//    pieces) and block scales into a raw ring;
//  * four convert warps widen them to f16 (exact: E4M3, and E2M1 times its
//    block scale, are f16 values) into two K and two V operand tiles in the
//    128-byte swizzle -- once for all of the CTA's rows.  Rows past the prefix
//    become zeros, so that nothing a page holds there reaches a result;
//  * one thread issues tcgen05 MMAs (f16, M = 128): S = Q K^T (K-major K tile)
//    and O += P V (the V tile read MN-major, P from tensor memory);
//  * two sets of four softmax warps, one row per thread (so a row's maximum and
//    sum need no shuffle), turn S into P in place: P's f16 pairs overwrite the
//    S columns already read.  Their slots alternate on the tensor pipe: two row
//    tiles with one K/V tile (MT = 2), or even and odd token tiles of one row
//    tile with accumulators of their own that are joined at the end (MT = 1).
// The query rows are prescaled by a power of two into f16 (kvq_device.cuh): the
// bf16 values are exact.  P is scaled by 2^7 against the row's (lazily moving)
// maximum and goes into the products as an f16 high part plus an f16 residual,
// like the decode kernel's, at twice the MMAs of one part.  A weight is off by
// 2^-22 of itself from 2^-10 of the reference on; below that the residual's step
// counts, 2^-32 of the row's largest weight for each token (a weight below that
// is in the sum and not in the products).  A caller that asks for it gets one
// part: 2^-11 of a weight from 2^-21 of the reference on, the same 2^-32 below
// (64 requests x 32k tokens, FP8: 60.2 us against 66.7 with two; NVFP4, 48 x 16k:
// 36.6 against 41.2; 4 x 1k: 11.1 against 12.2).  Sums and accumulators are
// fp32.
// Every wait is bounded; a timeout sets an error bit and the partials become
// NaN.
//
// What bounds it (FP8, head_dim 128, 256 rows x 8 heads over 32768 tokens in 12
// splits: 96 CTAs): a 128-token tile of both row tiles takes 2.2 us (the slope of
// the time from 4 to 8 splits), for which the products (2 x 3 of 128^3) need 1.5
// us at 2070 MHz; the rest is the chain scores -> maximum -> exponentials -> P V as
// far as the other slot does not cover it.  The kernel alone: 61.1 us, its SMs'
// tensor pipes active 60% of the time.  With one part and
// 11 splits clock stamps showed a tile every 3300 to 3500 cycles against 2048 of
// products, some 10000 cycles before the first scores, most of them until the
// queries have come, and 8000 from the last tile to the end (128 KB of partials per
// CTA), of 98000.  Measured slower (with one part): clusters that merge eight splits
// through distributed shared memory (4 requests x 1k: +4 us), the partials staged
// for bulk stores (64 x 32k: +0.8 us), P handed over whole (+0.1 to 0.4 us).

#include <cfloat>
#include <type_traits>

#include "kvq_attn.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kTok = 128;                 // tokens per tile
constexpr int kCol = kTok * 128;          // bytes of 64 f16 columns of 128 rows
constexpr int kConvWarp = 8;              // warps 0-7 softmax (slots 0, 1)
constexpr int kConvWarps = 4;
constexpr int kMmaWarp = kConvWarp + kConvWarps, kTmaWarp = kMmaWarp + 1, kReadyWarp = kTmaWarp + 1;
constexpr int kSharedThreads = 512;       // four warpgroups: softmax x 2, convert, MMA and TMA
// Registers per thread of the warpgroups (the launch gives each thread 128, 512
// for the four): a softmax thread holds its row's 128 scores at once.
constexpr int kRegSoft = 176, kRegConv = 96, kRegIssue = 64;
static_assert(2 * kRegSoft + kRegConv + kRegIssue <= 4 * 128, "register pool of the launch");
constexpr float kPShift = 7.0f;           // log2 scale of P
constexpr int kTmem = 512;                // S0 | S1 | O0 | O1, 128 columns each

template <int FMT, int D, int MT>
struct SharedGeom {
  using Gm = Geom<FMT, D>;
  static constexpr int kCols = D / 64;                  // 64-dim operand columns
  static constexpr int kTile = kCols * kCol;            // one f16 operand tile
  static constexpr int kRawCodes = kTok * Gm::kRow;
  static constexpr int kRaw = (kRawCodes + kTok * Gm::kSRow + 1023) / 1024 * 1024;
  static constexpr int kOffK = MT * kTile;              // Q tiles, then two K, two V
  static constexpr int kOffV = kOffK + 2 * kTile;
  static constexpr int kOffRaw = kOffV + 2 * kTile;
  // raw ring: as many K and V slots as fit, at most four
  static constexpr int kRoom = (229376 - kOffRaw) / (2 * kRaw);
  static constexpr int kSlots = kRoom < 4 ? kRoom : 4;
  static constexpr int kOffCtl = kOffRaw + 2 * kSlots * kRaw;
  static_assert(kSlots >= 1, "shared memory");
};

struct SharedCtl {
  uint64_t raw_full[2][4], raw_empty[2][4];   // [K, V][slot]
  uint64_t op_full[2][2], op_empty[2][2];     // [K, V][operand tile]
  uint64_t s_full[2], p_full[2][2], o_full[2];   // per softmax slot (P: per half of the tokens)
  uint64_t q_full, mma_done;
  uint32_t tmem;
  int abort_flag;
  float m[2][kTok], l[2][kTok];               // MT = 1: the slots' states
};

__device__ __forceinline__ void st_v8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The first of n lengths that is at least `least`, or -1 (a converged warp).  Out
// of line: it is rarely called, from a place that every copy waits for.
__device__ __noinline__ int first_as_long(const int32_t* lens, int n, int least) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = 0; i < n; i += 32) {
    const uint32_t m = __ballot_sync(0xffffffffu, i + lane < n && __ldg(lens + i + lane) >= least);
    if (m) return i + __ffs(m) - 1;
  }
  return -1;
}

template <int FMT, int D, int MT, bool P2>
__global__ void __launch_bounds__(kSharedThreads, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const SharedArgs a) {
  using Gm = Geom<FMT, D>;
  using Sg = SharedGeom<FMT, D, MT>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];   // the swizzle period
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(dyn_smem);
  SharedCtl& sm = *reinterpret_cast<SharedCtl*>(dyn_smem + Sg::kOffCtl);
  volatile int* abort_flag = &sm.abort_flag;

  if (warp == kTmaWarp && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < Sg::kSlots; ++k) {
        mbar_init(smem_u32(&sm.raw_full[i][k]), 1);
        mbar_init(smem_u32(&sm.raw_empty[i][k]), kConvWarps);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(smem_u32(&sm.op_full[i][k]), kConvWarps);
        mbar_init(smem_u32(&sm.op_empty[i][k]), 1);
      }
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      for (int k = 0; k < 2; ++k) mbar_init(smem_u32(&sm.p_full[i][k]), 4);
      mbar_init(smem_u32(&sm.o_full[i]), 1);
    }
    mbar_init(smem_u32(&sm.q_full), 4 * MT);
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
  // Every thread waits for the earlier work; the decode kernel, which may start
  // from here on and does not wait for this one, acquires that from the words
  // that the first CTA's spare warp publishes.
  griddep_wait();
  griddep_launch_dependents();

  const int h = blockIdx.y, split = blockIdx.z;
  const int row0 = blockIdx.x * (MT * kTok);
  // tiles [t0, t1) of the prefix
  const int tiles = (a.prefix + kTok - 1) / kTok;
  const int t0 = (int)((unsigned)split * (unsigned)tiles / (unsigned)a.splits);   // < 2^30
  const int t1 = (int)((unsigned)(split + 1) * (unsigned)tiles / (unsigned)a.splits);
  const int nt = t1 - t0;
  const int units = MT * nt;   // (slot, token tile) pairs in tensor-pipe order

  // Without a table of its own the prefix's pages are the first entries of the
  // first request that is as long: mostly request 0, whose entries are on their way
  // while its length is looked at.  Null: nobody shares, and no row takes anything
  // from what is read.  (Looking costs 4 x 1k 0.35 us of 11.85, 16 x 8k 0.3 of 20.1.)
  const int32_t* table = a.prefix_table ? a.prefix_table : a.block_table;
  if (warp == kTmaWarp && !a.prefix_table) {
    const int tok = min(t0 * kTok + lane * a.box, a.prefix - 1);
    asm volatile("prefetch.global.L1 [%0];" ::"l"(table + tok / a.ps));
    if (__ldg(a.seq_lens) < a.prefix) {
      const int first = first_as_long(a.seq_lens, a.batch, a.prefix);
      table = first < 0 ? nullptr : table + (size_t)first * a.max_pages;
    }
  }
  // TMA warp: lane i's cache row of box i (at most eight) of the split's tile j
  auto box_row = [&](int j) -> int {
    const int tok = (t0 + j) * kTok + lane * a.box;
    if (lane * a.box >= kTok || tok >= a.prefix || !table) return 0;
    const int pidx = tok / a.ps;
    int page = __ldg(table + pidx);
    if (page < 0 || page >= a.num_pages) {
      record_error(a.error_flag, 4);
      page = 0;
    }
    return (int)(((long)page * a.Hkv + h) * a.ps + (tok - pidx * a.ps));
  };
  // Softmax thread: its row (slot, r) of the kv head's query rows
  const int slot = (warp >> 2) & 1, r = threadIdx.x & (kTok - 1);
  const int row = row0 + (MT == 2 ? slot * kTok : 0) + r;
  const bool live = warp < kConvWarp && row < a.R;
  const int b = live ? row / a.G : 0, hq = h * a.G + (live ? row - b * a.G : 0);

  // The copies of tile j (TMA warp): K, then V, of row `row` of each lane's box
  auto copy_tile = [&](int j, int kv, int row) {
    const int nb = (min(kTok, a.prefix - (t0 + j) * kTok) + a.box - 1) / a.box;
    const int rs = j % Sg::kSlots;
    const uint32_t full = smem_u32(&sm.raw_full[kv][rs]);
    const uint32_t dst = base + Sg::kOffRaw + (2 * rs + kv) * Sg::kRaw;
    if (lane == 0) mbar_arrive_expect_tx(full, nb * a.box * (Gm::kRow + Gm::kSRow));
    __syncwarp();
    if (lane < nb) {
      tma_load_2d(dst + lane * a.box * Gm::kRow, kv ? &tmV : &tmK, 0, row, full);
      if constexpr (FMT == kFmtNvfp4)
        bulk_load(dst + Sg::kRawCodes + lane * a.box * Gm::kSRow,
                  (kv ? a.v_bscale : a.k_bscale) + (long)row * Gm::kSRow, a.box * Gm::kSRow,
                  full);
    }
  };

  // The first copies and the query loads go out before the CTA meets: they are
  // the longest steps to the first MMA.
  int len = 0;
  if (warp == kTmaWarp) {
    __syncwarp();   // lane 0 has set up the barriers: the others need not wait for more
    asm volatile("bar.arrive 3, %0;" ::"n"(kSharedThreads) : "memory");
    for (int j = 0; j < min(nt, Sg::kSlots); ++j) {
      const int row = box_row(j);
      copy_tile(j, 0, row);
      copy_tile(j, 1, row);
    }
  } else if (warp == kReadyWarp) {   // needs nothing of the CTA's set-up either
    asm volatile("bar.arrive 3, %0;" ::"n"(kSharedThreads) : "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
      publish_ready(a.ready, a.ready_n, lane);
  }
  // Queries.  Two row tiles: their 16-byte pieces go straight to the places of
  // the operand tile that their f16 values take, piece c of a row there, FP8
  // codes at 2c (they widen to 2c and 2c + 1); consecutive lanes copy
  // consecutive pieces, and rows past the last are zeros (64 requests x 32k
  // tokens, 256 rows, P in one part: 57.1 us against 59.0 with a row per thread,
  // whose loads touch 32 lines each).  One row tile: a row per thread in registers,
  // which is less code for the few rows (4 requests x 1k, one part: 10.2 us against
  // 10.9 staged).  (Plain copies and loads: queries may lie in pinned host memory.)
  const uint32_t qtile = base + (MT == 2 ? slot * Sg::kTile : 0);
  auto q_at = [&](int trow, int piece) -> uint32_t {
    return qtile + (piece >> 3) * kCol + (trow >> 3) * 1024 + (trow & 7) * 128 +
           (((piece ^ trow) & 7) << 4);
  };
  if (warp < kConvWarp) {
    if constexpr (MT == 2) {
      const int lp = a.q_fp8 ? D / 16 : D / 8;   // pieces of a row: a power of two
      const int c = lane & (lp - 1), per = 32 / lp;
      const int first = row0 + slot * kTok + 32 * (warp & 3) + lane / lp;
      // row first + k per: request qb, head qg of the group, without a division each
      int qb = first / a.G, qg = first - qb * a.G;
      const int db = per / a.G, dg = per - db * a.G;
      const long row_bytes = 16 * lp;
      const uint8_t* q0 = static_cast<const uint8_t*>(a.q) + (long)h * a.G * row_bytes + 16 * c;
#pragma unroll 4
      for (int k = 0; k < lp; ++k) {
        const int trow = 32 * (warp & 3) + lane / lp + k * per;
        const bool in = first + k * per < a.R;
        const uint8_t* src = in ? q0 + ((long)qb * a.Hq + qg) * row_bytes : q0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(
                         q_at(trow, a.q_fp8 ? 2 * c : c)),
                     "l"(src), "r"(in ? 16 : 0)
                     : "memory");
        qb += db;
        qg += dg;
        if (qg >= a.G) {
          qg -= a.G;
          ++qb;
        }
      }
    }
    len = live ? __ldg(a.seq_lens + b) : -1;
  }
  tc_fence_before();
  if (warp != kTmaWarp && warp != kReadyWarp)
    asm volatile("bar.sync 3, %0;" ::"n"(kSharedThreads) : "memory");
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (warp == kMmaWarp && tmem != 0) *abort_flag = 1;   // (never: all of it is ours)

  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
    if (wait_or_abort(smem_u32(&bar), parity, abort_flag)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp >= kMmaWarp) {
    regs_dec<kRegIssue>();
    if (warp == kTmaWarp) {
      // ================================================================= TMA
      int issued[2] = {min(nt, Sg::kSlots), min(nt, Sg::kSlots)};
      for (int j = Sg::kSlots; j < nt; ++j) {
        const int row = box_row(j);
        const int rs = j % Sg::kSlots;
        bool ok = true;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = __all_sync(0xffffffffu, wait(sm.raw_empty[kv][rs], (j / Sg::kSlots - 1) & 1));
          if (!ok) break;
          copy_tile(j, kv, row);
          issued[kv] = j + 1;
        }
        if (!ok) break;
      }
      // no copy in flight at exit (bounded waits)
      if (lane == 0)
        for (int kv = 0; kv < 2; ++kv)
          for (int j = max(0, issued[kv] - Sg::kSlots); j < issued[kv]; ++j)
            mbar_wait(smem_u32(&sm.raw_full[kv][j % Sg::kSlots]), (j / Sg::kSlots) & 1);
    } else if (warp == kMmaWarp) {
      // ================================================================= MMA
      // The warp stays converged, its elected lane issues; tensor memory
      // starts at column 0 (all of it is this CTA's).
      constexpr uint32_t kIdS = idesc(0, 0, 0, kTok), kIdO = idesc(0, 0, 1, D);
      const uint64_t dq = sdesc(base, 16, 1024);
      const uint64_t dk = sdesc(base + Sg::kOffK, 16, 1024);
      const uint64_t dv = sdesc(base + Sg::kOffV, kCol, 1024);   // MN-major
      auto wait_warp = [&](uint64_t& bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait(bar, parity));
      };
      bool ok = nt == 0 || wait_warp(sm.q_full, 0);
      // unit u: slot u & 1; token tile u / MT
      auto issue_s = [&](int u) {
        const int j = u / MT, slot = u & 1;
        // the first use of a K tile waits for it
        if (MT == 1 || slot == 0) ok = ok && wait_warp(sm.op_full[0][j & 1], (j >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t q = dq + (uint64_t)((MT == 2 ? slot : 0) * Sg::kTile >> 4);
        const uint64_t k = dk + (uint64_t)((j & 1) * Sg::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * kCol + (kk & 3) * 32) >> 4);
          mma_ss_elect(slot * 128, q + off, k + off, kIdS, kk > 0);
        }
        mma_commit_elect(smem_u32(&sm.s_full[slot]));
        if (MT == 1 || slot == 1) mma_commit_elect(smem_u32(&sm.op_empty[0][j & 1]));
      };
      for (int u = 0; u < min(2, units) && ok; ++u) issue_s(u);
      for (int u = 0; u < units && ok; ++u) {
        const int j = u / MT, slot = u & 1, i = u >> 1;   // the slot's i-th unit
        const uint64_t v = dv + (uint64_t)((j & 1) * Sg::kTile >> 4);
        const uint32_t p = slot * 128, o = 256 + slot * 128;
        if (MT == 1 || slot == 0) ok = wait_warp(sm.op_full[1][j & 1], (j >> 1) & 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // the halves of P, as they are written
          ok = ok && wait_warp(sm.p_full[slot][half], i & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k4 = 0; k4 < kTok / 32; ++k4) {
            const int kk = half * (kTok / 32) + k4;
            const uint64_t vk = v + (uint64_t)(kk * 2048 >> 4);
            if constexpr (P2) {   // high parts and residuals in alternating 16-column groups
              const uint32_t pk = p + 32 * (kk >> 1) + 8 * (kk & 1);
              mma_ts_elect(o, pk, vk, kIdO, i > 0 || kk > 0);
              mma_ts_elect(o, pk + 16, vk, kIdO, true);
            } else {
              mma_ts_elect(o, p + 8 * kk, vk, kIdO, i > 0 || kk > 0);
            }
          }
        }
        if (!ok) break;
        mma_commit_elect(smem_u32(&sm.o_full[slot]));
        if (MT == 1 || slot == 1) mma_commit_elect(smem_u32(&sm.op_empty[1][j & 1]));
        if (u + 2 < units) issue_s(u + 2);
      }
      // every MMA has completed at exit (bounded wait)
      mma_commit_elect(smem_u32(&sm.mma_done));
      mbar_wait(smem_u32(&sm.mma_done), 0);
      __syncwarp();
    }
  } else if (warp >= kConvWarp) {
    regs_dec<kRegConv>();
    // ============================================================= convert
    const int t = threadIdx.x - 32 * kConvWarp;
    const int p = t & 7, r = t;   // row r of the tile, row p of its 8-row atom
    for (int j = 0; j < nt; ++j) {
      const int rs = j % Sg::kSlots;
      const int nvalid = a.prefix - (t0 + j) * kTok;
      bool ok = true;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t raw = base + Sg::kOffRaw + (2 * rs + kv) * Sg::kRaw;
        const uint32_t dst = base + (kv ? Sg::kOffV : Sg::kOffK) + (j & 1) * Sg::kTile +
                             (r >> 3) * 1024 + p * 128;
        ok = wait(sm.raw_full[kv][rs], (j / Sg::kSlots) & 1);
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
            sc[c] = r < nvalid ? lds16(raw + Sg::kRawCodes + r * Gm::kSRow + 2 * c) : 0u;
        }
        // the operand tile was last read by the MMAs of tile j - 2
        if (j >= 2) ok = wait(sm.op_empty[kv][j & 1], ((j >> 1) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
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
            sts128(row + ((q ^ p) << 4), o[0], o[1], o[2], o[3]);
            sts128(row + (((q + 1) ^ p) << 4), o[4], o[5], o[6], o[7]);
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
              sts128(row + ((q ^ p) << 4), hmul2(e0, s), hmul2(e1, s), hmul2(e2, s),
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
      if (!__all_sync(0xffffffffu, ok)) break;
    }
  } else {
    regs_inc<kRegSoft>();
    // ============================================================= softmax
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t sS = lane_addr + slot * 128, sO = lane_addr + 256 + slot * 128;

    // ---- the row's query, into its operand tile
    // Score scale, log2 domain: positive, so that the row's largest score is that of
    // its largest product and the -inf past the prefix stays one.  A scale below
    // zero (a query head's) turns the query's sign instead; one of zero, also by
    // underflow (|q| below 2^-113), counts as the smallest normal number, whose
    // products with scores below 2^31 are nothing beside an exponent.
    float qsc;
    {
      // the largest magnitudes of a piece's even and odd bf16 values
      auto largest = [](const uint4& v) -> uint32_t {
        return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                        __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
      };
      uint32_t flip = 0u;   // sign bits of a pair, where the query's sign turns
      auto settle_scale = [&](float s) {
        if (s < 0.f) flip = 0x80008000u;
        qsc = s == 0.f ? FLT_MIN : fabsf(s);   // (NaN stays)
      };
      // bf16 piece c, prescaled by a power of two, as f16
      auto scale_piece = [&](const uint4& v, float f, int c) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k] = pack_f16x2(__uint_as_float(w[k] << 16) * f,
                            __uint_as_float(w[k] & 0xFFFF0000u) * f) ^ flip;
        sts128(q_at(r, c), o[0], o[1], o[2], o[3]);
      };
      // 16 FP8 codes as the f16 pieces 2c and 2c + 1
      auto widen_piece = [&](const uint4& v, int c) {
        uint32_t o[8];
        e4m3x4_to_f16x2x2(v.x, o[0], o[1]);
        e4m3x4_to_f16x2x2(v.y, o[2], o[3]);
        e4m3x4_to_f16x2x2(v.z, o[4], o[5]);
        e4m3x4_to_f16x2x2(v.w, o[6], o[7]);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] ^= flip;
        sts128(q_at(r, 2 * c), o[0], o[1], o[2], o[3]);
        sts128(q_at(r, 2 * c + 1), o[4], o[5], o[6], o[7]);
      };
      const float k_log2 =
          (a.k_hs ? a.sm_scale * __ldg(a.k_hs + h) : a.sm_scale * a.k_scale) * 1.4426950408889634f;
      if (a.q_fp8) settle_scale(k_log2 * (a.q_hs ? __ldg(a.q_hs + hq) : a.q_scale));
      if constexpr (MT == 2) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();   // the warp's rows are here
        if (a.q_fp8) {
#pragma unroll 2
          for (int c = 0; c < D / 16; ++c) widen_piece(lds128(q_at(r, 2 * c)), c);
        } else {
          uint32_t m2 = 0;
#pragma unroll 8
          for (int c = 0; c < D / 8; ++c) m2 = __vmaxu2(m2, largest(lds128(q_at(r, c))));
          const int e = q_prescale_exp(max(m2 & 0xFFFFu, m2 >> 16));
          settle_scale(scale_pow2(k_log2, -e));
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) scale_piece(lds128(q_at(r, c)), exp2i(e), c);
        }
      } else {
        const uint4* qp = reinterpret_cast<const uint4*>(
            static_cast<const uint8_t*>(a.q) + ((size_t)b * a.Hq + hq) * (a.q_fp8 ? D : 2 * D));
        uint4 v[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          v[c] = live && (c < D / 16 || !a.q_fp8) ? qp[c] : make_uint4(0u, 0u, 0u, 0u);
        if (a.q_fp8) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            if (slot == 0) widen_piece(v[c], c);
        } else {
          uint32_t m2 = 0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) m2 = __vmaxu2(m2, largest(v[c]));
          const int e = q_prescale_exp(max(m2 & 0xFFFFu, m2 >> 16));
          settle_scale(scale_pow2(k_log2, -e));
          if (slot == 0) {   // (both slots have the same rows)
#pragma unroll
            for (int c = 0; c < D / 8; ++c) scale_piece(v[c], exp2i(e), c);
          }
        }
      }
      if (MT == 2 || slot == 0) {
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full));
      }
    }

    // ---- the slot's units
    const int cnt = MT == 2 ? nt : (nt + 1 - slot) / 2;
    float m = -INFINITY, l = 0.f;   // reference max (log2), sum of 2^(x - m + 7)
    for (int i = 0; i < cnt; ++i) {
      const int j = MT == 2 ? i : 2 * i + slot;
      const int nvalid = a.prefix - (t0 + j) * kTok;
      if (!__all_sync(0xffffffffu, wait(sm.s_full[slot], i & 1))) break;
      tc_fence_after();
      uint32_t s[4][32];   // the row's scores
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(sS + 32 * c, s[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld32(s[c]);
      if (nvalid < kTok) {   // past the prefix
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (32 * c + k >= nvalid) s[c][k] = 0xFF800000u;   // -inf
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
          hi[k] = pack_f16x2(p0, p1);
          if constexpr (P2) {
            const float2 f = unpack_f16x2(hi[k]);
            lo[k] = pack_f16x2(p0 - f.x, p1 - f.y);
          }
        }
        tmem_st16(sS + (P2 ? 32 * c : 16 * c), hi);
        if constexpr (P2) tmem_st16(sS + 32 * c + 16, lo);
        if (c & 1) {   // half of P is written (and O rescaled): its MMAs may go
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[slot][c >> 1]));
        }
      }
      const float2 sum = unpack2(sum2);
      l += sum.x + sum.y;
    }

    // ---- the row's partial
    const bool share = live && len >= a.prefix;
    const float out_mult = a.v_hs ? __ldg(a.v_hs + h) : a.v_scale;
    const size_t prow = ((size_t)b * a.Hq + hq) * a.part_splits + a.split0 + split;
    if constexpr (MT == 1) {   // the other slot's state
      sm.m[slot][r] = m;
      sm.l[slot][r] = l;
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    const int cnt1 = nt / 2;   // MT = 1: units of slot 1
    bool done = true;
    if (MT == 2) {
      if (cnt > 0) done = wait(sm.o_full[slot], (cnt - 1) & 1);
    } else if (nt > 0) {
      done = wait(sm.o_full[0], (nt - 1 - cnt1) & 1);
      if (cnt1 > 0) done = wait(sm.o_full[1], (cnt1 - 1) & 1) && done;
    }
    const bool bad = __any_sync(0xffffffffu, !done || *abort_flag != 0);
    tc_fence_after();
    float f[2] = {0.f, 0.f};   // factors of the slots' accumulators
    float lse = -INFINITY;
    {
      const float m0 = MT == 1 ? sm.m[0][r] : m, l0 = MT == 1 ? sm.l[0][r] : l;
      const float m1 = MT == 1 ? sm.m[1][r] : -INFINITY, l1 = MT == 1 ? sm.l[1][r] : 0.f;
      const float M = fmaxf(m0, m1);
      const float e0 = m0 == -INFINITY ? 0.f : ex2(m0 - M), e1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
      const float L = e0 * l0 + e1 * l1;
      // l0, l1 may be NaN (a NaN or infinite score): it passes through
      if (M != -INFINITY && L != 0.f) {
        f[0] = e0 / L * out_mult;
        f[1] = e1 / L * out_mult;
        lse = (M - kPShift + log2f(L)) * kLn2;
      } else if (!(l0 == 0.f && l1 == 0.f)) {
        f[0] = f[1] = NAN;
        lse = NAN;
      }
    }
    lse = !share ? -INFINITY : bad ? NAN : lse;
    if (live && (MT == 2 || slot == 0)) a.part_lse[prow] = lse;
    // MT = 2: the slot's own O; MT = 1: both, half of the dims per slot
    constexpr int kChunks = MT == 2 ? D / 32 : D / 64;
    const int c0 = MT == 2 ? 0 : slot * kChunks;
    float* po = a.part_o + prow * D;
#pragma unroll 1
    for (int c = c0; c < c0 + kChunks; ++c) {
      uint32_t s[32];
      float o[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = 0.f;
      if (nt > 0 && !bad) {
        tmem_ld32(lane_addr + 256 + (MT == 2 ? slot * 128 : 0) + 32 * c, s);
        tmem_wait_ld32(s);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(s[k]) * f[0];
        if (MT == 1 && cnt1 > 0) {
          tmem_ld32(lane_addr + 256 + 128 + 32 * c, s);
          tmem_wait_ld32(s);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] += __uint_as_float(s[k]) * f[1];
        }
      }
      if (live) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = !share ? 0.f : bad ? NAN : o[8 * k + e];
          st_v8(po + 32 * c + 8 * k, v);
        }
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

// Merge of a row's partials (the arithmetic of the split merge: M = max lse,
// w_j = e^(lse_j - M), O = sum w_j o_j / sum w_j, 0 when all are empty), one
// warp per row: every partial is one coalesced read, eight in flight per lane.
constexpr int kMergeWarps = 8;

// 64 x 32 rows of 13 partials (14 MB): 9.2 us with cold caches, 1.5 TB/s and 12%
// of the issue slots: bound by the latency of its two rounds of reads.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_rows_kernel(const CombineArgs a) {
  constexpr int kPer = D / 32;   // dims per lane
  using Vec = std::conditional_t<kPer == 4, float4, float2>;
  griddep_wait();
  const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= a.rows) return;   // the whole warp
  const int s = a.num_splits;
  const float* lse = a.part_lse + (size_t)row * s;
  const Vec* po = reinterpret_cast<const Vec*>(a.part_o + (size_t)row * s * D) + lane;
  Vec v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < s) v[k] = __ldcg(po + k * 32);
  const float l0 = lane < s ? __ldcg(lse + lane) : -INFINITY;
  const float l1 = lane + 32 < s ? __ldcg(lse + lane + 32) : -INFINITY;
  float M = fmaxf(l0, l1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float e0 = l0 == -INFINITY ? 0.f : expf(l0 - M), e1 = l1 == -INFINITY ? 0.f : expf(l1 - M);
  float sum = e0 + e1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int j0 = 0; j0 < s; j0 += 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = j0 + k;
      const float w = __shfl_sync(0xffffffffu, j < 32 ? e0 : e1, j & 31);
      if (j < s) {
        const float* f = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += w * f[i];
        if (j + 8 < s) v[k] = __ldcg(po + (j + 8) * 32);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] *= inv;
  const size_t at = (size_t)row * D + lane * kPer;
  if (a.out_dtype == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) store_out_t<0>(a.out, a.out_scale, at + i, acc[i]);
  } else if (a.out_dtype == 1) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) store_out_t<1>(a.out, a.out_scale, at + i, acc[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) store_out_t<2>(a.out, a.out_scale, at + i, acc[i]);
  }
}

// Runs `f` with the kernel of these types and its shared memory.
template <typename F>
cudaError_t with_kernel(int fmt, int D, int R, int wide_p, F&& f) {
  auto pick = [&](auto kfmt, auto kd, auto mt, auto p2) {
    constexpr int FMT = decltype(kfmt)::value, DD = decltype(kd)::value;
    constexpr int MT = decltype(mt)::value;
    using Sg = SharedGeom<FMT, DD, MT>;
    constexpr size_t smem = Sg::kOffCtl + sizeof(SharedCtl);
    static_assert(smem <= 232448, "shared memory of one CTA");
    return f(shared_prefix_kernel<FMT, DD, MT, decltype(p2)::value>, smem, MT);
  };
  auto by_p = [&](auto kfmt, auto kd, auto mt) {
    return wide_p ? pick(kfmt, kd, mt, std::true_type{}) : pick(kfmt, kd, mt, std::false_type{});
  };
  // Up to 128 rows one row tile with token tiles in both slots, else two row
  // tiles (16 x 8k, 64 rows: 20.5 us against 25.3 with two; 64 x 32k, 256 rows:
  // 67.3 against 83.7 with one).
  auto by_rows = [&](auto kfmt, auto kd) {
    return R > kTok ? by_p(kfmt, kd, std::integral_constant<int, 2>{})
                    : by_p(kfmt, kd, std::integral_constant<int, 1>{});
  };
  using Fp8 = std::integral_constant<int, kFmtFp8>;
  using Nvfp4 = std::integral_constant<int, kFmtNvfp4>;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (fmt == kFmtFp8 && D == 128) return by_rows(Fp8{}, D128{});
  if (fmt == kFmtFp8 && D == 64) return by_rows(Fp8{}, D64{});
  if (fmt == kFmtNvfp4 && D == 128) return by_rows(Nvfp4{}, D128{});
  if (fmt == kFmtNvfp4 && D == 64) return by_rows(Nvfp4{}, D64{});
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_merge_rows(const CombineArgs& a, cudaStream_t st) {
  const dim3 grid((a.rows + kMergeWarps - 1) / kMergeWarps), block(32 * kMergeWarps);
  if (a.num_splits > kMaxFusedSplits) return cudaErrorInvalidValue;
  if (a.Dv == 128) return launch_pdl(merge_rows_kernel<128>, grid, block, 0, st, a);
  if (a.Dv == 64) return launch_pdl(merge_rows_kernel<64>, grid, block, 0, st, a);
  return cudaErrorInvalidValue;
}

cudaError_t launch_shared_prefix(int fmt, int D, const TensorMaps& m, const SharedArgs& a,
                                 cudaStream_t st) {
  return with_kernel(fmt, D, a.R, a.wide_p, [&](auto kern, size_t smem, int mt) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((a.R + mt * kTok - 1) / (mt * kTok), a.Hkv, a.splits);
    return launch_pdl(kern, grid, dim3(kSharedThreads), smem, st, m.k16, m.v16, a);
  });
}

}  // namespace kvq
