// A step's paging on the GPU: new lengths, block-table entries, packed offsets,
// slots and positions of the new tokens, and the stack of free pages, from the
// requests' lengths and their changes (sm_103a).
//
// All of it is prefix sums over the requests.  With t_b new tokens, h_b pages held
// before and w_b wanted after, request b's tokens start at sum t, the pages that it
// returns (h > w) are the (sum of earlier returns)-th ones pushed, and the pages that
// it takes (w > h) the (sum of earlier takes)-th ones popped; a request is served
// where the takes up to its own end do not pass what the stack holds after all
// returns.  Every CTA forms the sums for all requests (two int32 per request, from
// L2) and then does its share of the tokens, returns and takes, finding an item's
// request by a binary search in shared memory.  No item reads what another writes:
// a popped page that was pushed in the same call is read where it came from, the
// block table's row of the request that returned it.  Only the lengths and the count
// may be updated in place, so the CTA that arrives last writes them.
//
// Bound by latency: the chain count and lengths -> two block scans -> search -> page
// -> slot.  256 requests with a token each 4.2 us, 1500 requests with 104000 tokens in
// mixed chunks 9.4 us (an empty kernel takes 0.7).

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// Threads: the requests' sums meet at fewer barriers in small blocks, and large batches
// have several requests per thread otherwise.
constexpr int kPlanSmall = 256, kPlanLarge = 1024;
constexpr int kTokensEach = 1;   // per thread, before another CTA is added (two: 10.7 us against 9.2 for 104000)

template <int T>
struct PlanSmem {
  long warp_a[T / 32], warp_b[T / 32];
  int pops, last;
};

// Exclusive sums of a and b over the block's threads, and their totals.
template <int T>
__device__ __forceinline__ void scan2(long& a, long& b, long& total_a, long& total_b,
                                      PlanSmem<T>& sm) {
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
  a -= a0;
  b -= b0;
  // the other warps' sums: a lane each
  long x = lane < T / 32 ? sm.warp_a[lane] : 0, y = lane < T / 32 ? sm.warp_b[lane] : 0;
  const long x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < T / 32; o <<= 1) {
    const long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  total_a = __shfl_sync(0xffffffffu, x, T / 32 - 1);
  total_b = __shfl_sync(0xffffffffu, y, T / 32 - 1);
  a += __shfl_sync(0xffffffffu, x - x0, warp);
  b += __shfl_sync(0xffffffffu, y - y0, warp);
  __syncthreads();   // (the sums' places may be written again)
}

// The last of n (>= 1) non-decreasing entries that is at most x (the first is).
__device__ __forceinline__ int owner(const int* first, int n, int x) {
  int lo = 0, hi = n;   // first[lo] <= x < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int clamp_int(long x) { return (int)min(x, (long)INT32_MAX); }

template <int T>
__global__ void __launch_bounds__(T) plan_kernel(const PlanArgs a) {
  extern __shared__ int dyn[];
  __shared__ PlanSmem<T> sm;
  const int B = a.batch, tid = threadIdx.x;
  int* tok0 = dyn;              // first new token of each request, clipped to max_tokens
  int* take0 = tok0 + B + 1;    // pages taken by the requests before
  int* back0 = take0 + B;       // pages returned by the requests before
  int* held = back0 + B;        // pages held before (a request that shrinks: after)
  int* old = held + B;          // length before; -1 - length: refused
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) sm.pops = 0;
  const bool report = blockIdx.x == 0;
  int err = 0;

  int count = *a.free_count;
  if (count < 0 || count > a.num_pages) {
    err |= kErrPool;
    count = count < 0 ? 0 : a.num_pages;
  }
  const int cap = a.max_pages * a.ps;   // (< 2^31)
  // x / page size, and the pages of x tokens, for 0 <= x < 2^31
  auto over_ps = [&](int x) -> int {
    return (int)((__umulhi((unsigned)x, a.ps_mul) + (unsigned)x) >> a.ps_shift);
  };
  auto pages = [&](int x) -> int { return x > 0 ? over_ps(x - 1) + 1 : 0; };
  const int per = (B + T - 1) / T;   // consecutive requests per thread
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);

  // ---- tokens and returned pages before each request
  long tokens = 0, back = 0;
  for (int b = b0; b < b1; ++b) {
    int l = a.seq_lens[b];
    const int d = a.add_lens[b];
    if (l < 0 || l > cap) {
      err |= 2;
      l = l < 0 ? 0 : cap;
    }
    old[b] = l;
    const int h = pages(l), w = d < 0 ? pages(d < -l ? 0 : l + d) : h;
    held[b] = w;
    tok0[b] = max(d, 0);        // (the counts, until the sums are known)
    back0[b] = h - w;
    take0[b] = d <= 0 ? 0 : d <= cap - l ? pages(l + d) - h : -1;   // -1: past its row
    tokens += max(d, 0);
    back += back0[b];
  }
  long all_tokens, all_back;
  scan2<T>(tokens, back, all_tokens, all_back, sm);
  if ((long)count + all_back > a.num_pages) err |= kErrPool;
  const int top = (int)min((long)count + all_back, (long)a.num_pages);   // after all returns

  // ---- pages taken before each request
  long take = 0, none = 0, all_take, unused;
  for (int b = b0; b < b1; ++b) {
    const int t = tok0[b], r = back0[b];
    if (t > 0 && (take0[b] < 0 || tokens + t > a.max_tokens)) {
      old[b] = -1 - old[b];
      take0[b] = 0;
    }
    tok0[b] = (int)min(tokens, (long)a.max_tokens);
    back0[b] = clamp_int(back);
    tokens += t;
    back += r;
    take += take0[b];
  }
  scan2<T>(take, none, all_take, unused, sm);
  int pops = 0;
  for (int b = b0; b < b1; ++b) {
    const int need = take0[b];
    take0[b] = clamp_int(take);
    take += need;
    if (need > 0) {
      if (take <= top) pops = (int)take;
      else old[b] = -1 - old[b];
    }
    if (old[b] < 0) err |= kErrRefused;
  }
  if (pops > 0) atomicMax(&sm.pops, pops);
  if (tid == 0) tok0[B] = (int)min(all_tokens, (long)a.max_tokens);
  if (err && report) record_error(a.error_flag, err);
  __syncthreads();
  pops = sm.pops;

  // The lengths and the count, by the CTA that arrives last: all others have read
  // theirs.
  if (tid == 0) {
    unsigned prev = 0;
    if (gridDim.x > 1)
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                   : "=r"(prev)
                   : "l"(a.counter)
                   : "memory");
    sm.last = prev == gridDim.x - 1;
    if (sm.last && gridDim.x > 1) *a.counter = 0u;
  }
  __syncthreads();
  if (sm.last) {
    for (int b = tid; b < B; b += T) {
      const int o = old[b], d = a.add_lens[b];
      a.seq_lens_out[b] = o < 0 ? -1 - o : (int)max((long)o + d, 0l);
    }
    if (tid == 0) *a.free_count_out = top - pops;
  }
  if (blockIdx.x == 0) {
    if (a.start_pos)
      for (int b = tid; b < B; b += T) a.start_pos[b] = old[b] < 0 ? -1 - old[b] : old[b];
    if (a.q_offsets)
      for (int b = tid; b <= B; b += T) a.q_offsets[b] = tok0[b];
  }

  // ---- this CTA's share of the items
  const int stride = gridDim.x * T, first = blockIdx.x * T + tid;
  const int pushes = top - count;
  auto in_range = [&](int page) -> bool {
    if (page >= 0 && page < a.num_pages) return true;
    record_error(a.error_flag, 4);
    return false;
  };
  auto pushed = [&](int r) -> int {   // the r-th returned page
    const int b = owner(back0, B, r);
    return a.block_table[(size_t)b * a.max_pages + held[b] + (r - back0[b])];
  };
  auto taken = [&](int g) -> int {    // the g-th page from the stack's top
    const int i = top - 1 - g;
    return i < count ? a.free_pages[i] : pushed(i - count);
  };
  for (int r = first; r < pushes; r += stride) {
    const int page = pushed(r);
    in_range(page);
    a.free_pages[count + r] = page;
  }
  for (int g = first; g < pops; g += stride) {
    const int b = owner(take0, B, g), page = taken(g);
    in_range(page);   // (where neither slots nor positions are wanted, nobody else looks)
    a.block_table[(size_t)b * a.max_pages + held[b] + (g - take0[b])] = page;
  }
  if (!a.slots && !a.positions) return;
  const int live = tok0[B];
  for (int i = first; i < a.max_tokens; i += stride) {
    long slot = -1;
    int pos = -1;
    if (i < live) {
      const int b = owner(tok0, B, i);
      if (old[b] >= 0) {
        pos = old[b] + (i - tok0[b]);
        const int p = over_ps(pos);
        const int page = p < held[b] ? a.block_table[(size_t)b * a.max_pages + p]
                                     : taken(take0[b] + (p - held[b]));
        if (in_range(page)) slot = (long)page * a.ps + (pos - p * a.ps);
      }
    }
    if (a.slots) a.slots[i] = slot;
    if (a.positions) a.positions[i] = pos;
  }
}

template <int T>
cudaError_t launch_t(const PlanArgs& a, cudaStream_t st) {
  constexpr size_t kMost = (5 * (size_t)kMaxPlanBatch + 1) * sizeof(int);
  static_assert(kMost + sizeof(PlanSmem<T>) <= 232448, "shared memory of one CTA");
  cudaError_t e = cudaFuncSetAttribute(plan_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kMost);
  if (e != cudaSuccess) return e;
  const size_t smem = (5 * (size_t)a.batch + 1) * sizeof(int);
  const long ctas = ((long)a.max_tokens + T * kTokensEach - 1) / (T * kTokensEach);
  const dim3 grid((unsigned)(ctas < 1 ? 1 : ctas > 152 ? 152 : ctas));
  return launch_pdl(plan_kernel<T>, grid, dim3(T), smem, st, a);
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st) {
  return a.batch <= kPlanSmall ? launch_t<kPlanSmall>(a, st) : launch_t<kPlanLarge>(a, st);
}

}  // namespace kvq
