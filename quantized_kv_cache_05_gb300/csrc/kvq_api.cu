// The extern "C" entry points of include/kvq.h: argument validation (before
// any launch), TMA descriptor setup and kernel dispatch.  Host code only.

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cudaTypedefs.h>

#include "kvq.h"
#include "kvq_internal.h"

using namespace kvq;

namespace {

bool finite_pos(float x) { return std::isfinite(x) && x > 0.f; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  // The CUDA driver API entry point is looked up once per process.
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Encodes a map of bytes with dense boxes (the arguments of
// cuTensorMapEncodeTiled).  The driver's call wants a current context, which a
// thread that has made no runtime call with one has not: it gets the device's.
bool encode_map(CUtensorMap* m, cuuint32_t rank, const void* base, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  int dev = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess &&
      cudaSetDevice(dev) == cudaSuccess)
    r = encode();
  return r == CUDA_SUCCESS;
}

// 2-D byte view [rows][row_bytes] of a cache tensor, box_rows-row boxes, with the
// widest hardware swizzle the row allows.
bool make_row_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows,
                  uint32_t box_rows = kBoxTokens) {
  cuuint64_t dims[2] = {row_bytes, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {(cuuint32_t)row_bytes, box_rows};
  CUtensorMapSwizzle sw = row_bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                          : row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : CU_TENSOR_MAP_SWIZZLE_NONE;
  return encode_map(m, 2, base, dims, strides, box, sw);
}

// 3-D byte view [rows][n_slices][slice_bytes] of a row-major tensor whose rows
// are n_slices * slice_bytes wide; boxes of one slice x box_rows rows.
bool make_slice_map(CUtensorMap* m, const void* base, uint64_t slice_bytes, uint64_t n_slices,
                    uint64_t rows, CUtensorMapSwizzle sw, uint32_t box_rows = kBoxTokens) {
  cuuint64_t dims[3] = {slice_bytes, n_slices, rows};
  cuuint64_t strides[2] = {slice_bytes, slice_bytes * n_slices};
  cuuint32_t box[3] = {(cuuint32_t)slice_bytes, 1, box_rows};
  return encode_map(m, 3, base, dims, strides, box, sw);
}

bool is_mla(const kvq_cache* c) { return c->rope_dim > 0; }

// Checks shared by append and decode.
kvq_status check_cache(const kvq_cache* c) {
  if (!c) return KVQ_ERR_INVALID;
  if (c->fmt != KVQ_FP8_E4M3 && c->fmt != KVQ_NVFP4) return KVQ_ERR_INVALID;
  if (c->num_pages < 1 || c->num_kv_heads < 1 || c->max_pages_per_seq < 1) return KVQ_ERR_INVALID;
  if (c->page_size < 16 || c->page_size % 16 != 0) return KVQ_ERR_INVALID;
  if (c->head_dim < 16 || c->head_dim % 16 != 0 || c->head_dim > 1024) return KVQ_ERR_INVALID;
  if ((long long)c->num_pages * c->num_kv_heads * c->page_size >= (1LL << 31))
    return KVQ_ERR_UNSUPPORTED;
  if (!c->block_table || !c->k_codes || !aligned16(c->k_codes)) return KVQ_ERR_INVALID;
  if (!c->k_head_scale && !finite_pos(c->k_scale)) return KVQ_ERR_INVALID;
  if (c->fmt == KVQ_NVFP4 && (!c->k_bscale || !aligned16(c->k_bscale))) return KVQ_ERR_INVALID;
  if (is_mla(c)) {
    if (c->rope_dim % 8 != 0 || !c->k_pe || !aligned16(c->k_pe)) return KVQ_ERR_INVALID;
    if (c->v_codes || !c->v_is_k_latent) return KVQ_ERR_INVALID;
    if (c->k_head_scale || c->v_head_scale) return KVQ_ERR_INVALID;
    if (c->num_kv_heads != 1) return KVQ_ERR_INVALID;
    if (c->fmt != KVQ_NVFP4) return KVQ_ERR_UNSUPPORTED;
  } else {
    if (c->rope_dim != 0 || c->k_pe || c->v_is_k_latent) return KVQ_ERR_INVALID;
    if (!c->v_codes || !aligned16(c->v_codes)) return KVQ_ERR_INVALID;
    if (!c->v_head_scale && !finite_pos(c->v_scale)) return KVQ_ERR_INVALID;
    if (c->fmt == KVQ_NVFP4 && (!c->v_bscale || !aligned16(c->v_bscale))) return KVQ_ERR_INVALID;
  }
  return KVQ_OK;
}

kvq_status check_params(const kvq_decode_params* p) {
  if (!p) return KVQ_ERR_INVALID;
  if (p->batch < 0 || p->num_q_heads < 1 || p->qk_dim < 1 || p->v_dim < 1) return KVQ_ERR_INVALID;
  if (p->num_splits < 1) return KVQ_ERR_INVALID;
  if (p->num_splits > kMaxFusedSplits) return KVQ_ERR_UNSUPPORTED;
  if (p->max_kv_len < 0) return KVQ_ERR_INVALID;
  if (p->batch > 0 && !p->seq_lens) return KVQ_ERR_INVALID;
  if (!finite_pos(p->sm_scale)) return KVQ_ERR_INVALID;
  if (!std::isfinite(p->prob_scale) || p->prob_scale < 0.f) return KVQ_ERR_INVALID;
  if (p->out_dtype < KVQ_OUT_F32 || p->out_dtype > KVQ_OUT_E4M3) return KVQ_ERR_INVALID;
  if (p->out_dtype == KVQ_OUT_E4M3 && !finite_pos(p->out_scale)) return KVQ_ERR_INVALID;
  if (p->fresh_tokens < 0) return KVQ_ERR_INVALID;
  if (p->q_fp8 != 0 && p->q_fp8 != 1) return KVQ_ERR_INVALID;
  if (p->q_fp8 && !p->q_head_scale && !finite_pos(p->q_scale)) return KVQ_ERR_INVALID;
  return KVQ_OK;
}

kvq_status check_diff(const kvq_diff* d) {
  if (!d || !d->lambda || !std::isfinite(d->gain)) return KVQ_ERR_INVALID;
  if (d->norm && (!aligned16(d->norm) || !(std::isfinite(d->eps) && d->eps >= 0.f)))
    return KVQ_ERR_INVALID;
  return KVQ_OK;
}

// Heads, dims and lengths of an attention call against the cache (not MLA); what
// else its kernels need, the caller checks.
kvq_status check_heads_of(const kvq_cache* c, const kvq_decode_params* p, bool wide) {
  const int D = c->head_dim;
  if (p->num_q_heads % c->num_kv_heads != 0 || p->qk_dim != D || p->v_dim != D)
    return KVQ_ERR_INVALID;
  if ((long long)p->max_kv_len > (long long)c->max_pages_per_seq * c->page_size)
    return KVQ_ERR_INVALID;
  if (D != 64 && D != 128 && !(wide && D == 256 && c->fmt == KVQ_NVFP4))
    return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

// Rows of heads, `tokens` of them: 16-byte loads need the base and the strides
// aligned; outputs may not overlap themselves.
kvq_status check_heads(const kvq_heads* h, int dim, long long tokens, bool out) {
  if (!h || !h->data || !aligned16(h->data) || h->num_heads < 1) return KVQ_ERR_INVALID;
  const long long ts = h->token_stride, hs = h->head_stride;
  if (ts < 0 || hs < 0 || ts % 8 != 0 || hs % 8 != 0) return KVQ_ERR_INVALID;
  if (ts >= (1LL << 31) || hs >= (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  if (out) {
    const bool by_token = (h->num_heads == 1 || hs >= dim) &&
                          (tokens == 1 || ts >= (h->num_heads - 1) * hs + dim);
    const bool by_head = (tokens == 1 || ts >= dim) &&
                         (h->num_heads == 1 || hs >= (tokens - 1) * ts + dim);
    if (!by_token && !by_head) return KVQ_ERR_INVALID;
  }
  return KVQ_OK;
}

kvq_status check_rotary(const kvq_rotary* r, int dim) {
  if (!r) return KVQ_ERR_INVALID;
  if (r->rot_dim < 0 || r->rot_dim > dim || r->rot_dim % 2 != 0) return KVQ_ERR_INVALID;
  if (r->interleaved != 0 && r->interleaved != 1) return KVQ_ERR_INVALID;
  if (r->rot_dim > 0 && (!r->cos_sin || !aligned16(r->cos_sin) || r->num_positions < 1))
    return KVQ_ERR_INVALID;
  if ((r->q_norm && !aligned16(r->q_norm)) || (r->k_norm && !aligned16(r->k_norm)))
    return KVQ_ERR_INVALID;
  if ((r->q_norm || r->k_norm) && !(std::isfinite(r->eps) && r->eps >= 0.f))
    return KVQ_ERR_INVALID;
  if (r->rot_dim % 32 != 0) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

// The query rows of a call: their output rows and E4M3 scale.
kvq_status check_query_rows(const kvq_heads* q, const kvq_heads* out, int dim, long long tokens,
                            int q_fp8, float q_scale, const float* q_head_scale) {
  kvq_status s = check_heads(q, dim, tokens, false);
  if (s != KVQ_OK) return s;
  s = check_heads(out, dim, tokens, true);
  if (s != KVQ_OK) return s;
  if (out->num_heads != q->num_heads) return KVQ_ERR_INVALID;
  if (q_fp8 != 0 && q_fp8 != 1) return KVQ_ERR_INVALID;
  if (q_fp8 && !q_head_scale && !finite_pos(q_scale)) return KVQ_ERR_INVALID;
  return KVQ_OK;
}

RopeRows rope_rows(const kvq_heads* h) {
  if (!h) return RopeRows{nullptr, 0, 0, 0};
  return RopeRows{static_cast<uint16_t*>(h->data), (long)h->token_stride, (long)h->head_stride,
                  h->num_heads};
}

void rotary_args(RopeArgs& a, const kvq_rotary* r) {
  a.cos_sin = r->cos_sin;
  a.num_positions = r->num_positions;
  a.rot = r->rot_dim;
  a.interleaved = r->interleaved;
  a.eps = r->eps;
}

// Row tiles of a kv head in the shared prefix's kernel: 128 query rows, or 256
// when there are more.
long long shared_row_tiles(long long batch, int q_per_kv) {
  const long long rows = batch * q_per_kv;
  return rows > 128 ? (rows + 255) / 256 : 1;
}

// x / d for 0 <= x < 2^31 as (umulhi(x, mul) + x) >> shift: with 2^(k-1) < d <= 2^k and
// mul = floor(2^32 (2^k - d) / d) + 1, the multiplier 2^32 + mul is above 2^(32+k) / d by at
// most one, so that the quotient's excess, x / 2^(32+k), stays below 1 / d.
void divisor(int d, uint32_t* mul, uint32_t* shift) {
  uint32_t k = 0;
  while ((1u << k) < (unsigned)d) ++k;
  *shift = k;
  *mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << k) - d)) / d + 1);
}

// TMA boxes of a 128-token tile: the largest power of two up to it that divides the pages.
int box_rows(int page_size) {
  int box = 16;
  while (box < 128 && page_size % (2 * box) == 0) box *= 2;
  return box;
}

// Workspace of kvq_chunk_attention: that of the chunks' kernels, then the counters and
// partials of the decode that takes the requests with a single new token (splits 0: there
// is none).  The decode reads a request's keys once for up to 16 query rows, in one
// launch with its own split; as row tiles of 128 those few rows cost as much as full
// ones (28 single tokens beside 4 chunks, NVFP4: 268 us, 240 with it).  A lone
// request is never worth its launch.  Where the batch fills the GPU anyway, kManyChunks
// chunks of each request at most: how long the requests are is known on the GPU only, and
// max_kv_len may be far more (256 requests of 1000 tokens, max_kv_len 131072, 8 kv heads: 229
// us and 57 MB with 4 chunks, 2106 us and 311 MB with the 64 of kvq_auto_splits); far longer
// requests than the others are not the decode's (kLongChunk).
constexpr int kManyChunks = 4;
struct ChunkParts {
  int splits;
  size_t counters, lse, o, bytes;
};
ChunkParts chunk_parts(int sms, const kvq_cache* c, const kvq_decode_params* p, const kvq_diff* d) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  ChunkParts w{};
  const int D = c->head_dim, rows = (d ? 2 : 1) * (p->num_q_heads / c->num_kv_heads);
  w.counters = up(chunk_workspace_bytes(sms, std::max(p->batch, 1), D));
  w.bytes = w.counters;
  // (NVFP4, one kv head and 16 rows would be taken for MLA there, whose kernel has one CTA on
  // an SM; 15 rows are this one's as well)
  if (p->batch < 2 || rows > kMaxGroup ||
      kvq_auto_splits(sms, p->batch, c->num_kv_heads, std::min(rows, kMaxGroup - 1), p->max_kv_len,
                      c->fmt, &w.splits) != KVQ_OK)
    return w;
  if ((long long)p->batch * c->num_kv_heads > 2 * sms) w.splits = std::min(w.splits, kManyChunks);
  const size_t groups = (size_t)p->batch * c->num_kv_heads, parts = groups * rows * w.splits;
  w.lse = w.counters + up(groups * sizeof(uint32_t));
  w.o = w.lse + up(parts * sizeof(float));
  w.bytes = w.o + parts * D * sizeof(float);
  return w;
}

kvq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

// kvq_rope_append and kvq_rope_append_slots: `where` says where the tokens go.
kvq_status rope_append(const kvq_cache* c, const kvq_rotary* r, long long tokens, const kvq_heads* k,
                       const kvq_heads* v, const kvq_heads* kpe, const kvq_heads* q,
                       const kvq_heads* q_out, int q_fp8, float q_scale, const float* q_head_scale,
                       int32_t* error_flag, const RopeArgs& where, cudaStream_t stream) {
  kvq_status s = check_cache(c);
  if (s != KVQ_OK) return s;
  if (tokens < 0) return KVQ_ERR_INVALID;
  const bool mla = is_mla(c);
  const int D = c->head_dim;
  s = check_rotary(r, mla ? c->rope_dim : D);
  if (s != KVQ_OK) return s;
  if (mla) {
    if (v || !kpe) return KVQ_ERR_INVALID;
    if (D != 512 || c->rope_dim != 64 || q) return KVQ_ERR_UNSUPPORTED;
  } else {
    if (!v || kpe) return KVQ_ERR_INVALID;
    if (D != 64 && D != 128 && D != 256) return KVQ_ERR_UNSUPPORTED;
  }
  if (tokens == 0) return KVQ_OK;
  if (!where.start_pos && !where.slots) return KVQ_ERR_INVALID;
  if (where.slots && r->rot_dim > 0 && !where.positions) return KVQ_ERR_INVALID;
  s = check_heads(k, D, tokens, false);
  if (s == KVQ_OK) s = mla ? check_heads(kpe, c->rope_dim, tokens, false)
                           : check_heads(v, D, tokens, false);
  if (s != KVQ_OK) return s;
  if (k->num_heads != c->num_kv_heads || (mla ? kpe : v)->num_heads != c->num_kv_heads)
    return KVQ_ERR_INVALID;
  if (q) {
    s = check_query_rows(q, q_out, D, tokens, q_fp8, q_scale, q_head_scale);
    if (s != KVQ_OK) return s;
  }
  const long long heads = mla ? 1 : 2LL * c->num_kv_heads + (q ? q->num_heads : 0);
  if (tokens >= (1LL << 31) || tokens * heads >= (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  RopeArgs a = where;
  a.fmt = c->fmt;
  rotary_args(a, r);
  a.q = rope_rows(q);
  a.k = rope_rows(k);
  a.v = rope_rows(mla ? kpe : v);
  a.q_out = rope_rows(q ? q_out : nullptr);
  a.q_norm = q ? r->q_norm : nullptr;
  a.k_norm = r->k_norm;
  a.tokens = (unsigned)tokens;
  a.q_fp8 = q ? q_fp8 : 0;
  a.q_scale = q_scale;
  a.q_recip = a.q_fp8 && !q_head_scale ? (float)(1.0 / (double)q_scale) : 0.f;
  a.q_hs = q_head_scale;
  a.error_flag = error_flag;
  a.Hkv = c->num_kv_heads;
  a.ps = c->page_size;
  a.max_pages = c->max_pages_per_seq;
  a.num_pages = c->num_pages;
  a.block_table = c->block_table;
  a.k_codes = static_cast<uint8_t*>(c->k_codes);
  a.v_codes = static_cast<uint8_t*>(c->v_codes);
  a.k_bscale = static_cast<uint8_t*>(c->k_bscale);
  a.v_bscale = static_cast<uint8_t*>(c->v_bscale);
  a.k_pe = static_cast<uint16_t*>(c->k_pe);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.k_recip = (float)(1.0 / (double)c->k_scale);
  a.v_recip = mla ? a.k_recip : (float)(1.0 / (double)c->v_scale);
  a.k_hs = c->k_head_scale;
  a.v_hs = c->v_head_scale;
  return cuda_status(launch_rope(D, mla, a, stream));
}

// ---------------------------------------------------------------------------
// Division by the prob scale (FP8 probabilities, vLLM PR 15734: softmax(QK^T)
// quantized to FP8 with prob_output_scale).  The kernels need E4M3(fl32(p /
// y)) for p in [0, 1] and the call's y = prob_scale.  With z = RN(1/y), the
// device's prob_quotient (q0 = RN(p z), r = RN(p - q0 y), q = RN(q0 + r z))
// is within one fp32 step of RN(p/y) for every p, and equals it unless p/y
// lies within about 2^-45 (relative) of the midpoint of two fp32 numbers.
// Two adjacent fp32 numbers can round to different E4M3 codes only if one of
// them is itself a rounding boundary of the E4M3 grid (a midpoint between two
// E4M3 values: every such midpoint is an fp32 number).  So the codes of the
// fast path equal those of the IEEE division for all p as soon as they do for
// every p whose quotient lies within 1.5 fp32 steps of a boundary; the check
// below runs the fast path on all p in a wider window (relative 2^-20) around
// each boundary's preimage and requires the correctly rounded quotient there.
// It is exact host arithmetic (this file is compiled with FP contraction off:
// the product and the two fused multiply-adds are the device's operations).
// ---------------------------------------------------------------------------

float fast_quotient(float p, float y, float z) {
  const float q0 = p * z;
  const float r = std::fma(-q0, y, p);
  return std::fma(r, z, q0);
}

// RN(p / y) in fp32: the double quotient is correctly rounded to 53 bits, and
// rounding it to 24 bits gives the correctly rounded fp32 quotient (53 >= 2 *
// 24 + 2).
float exact_quotient(float p, float y) { return (float)((double)p / (double)y); }

// Positive finite E4M3 values in increasing order (codes 0x00..0x7E).
double e4m3_positive(int code) {
  const int e = code >> 3, m = code & 7;
  return e == 0 ? std::ldexp((double)m, -9) : std::ldexp(1.0 + m / 8.0, e - 7);
}

bool prob_reciprocal_ok(float y, float* z_out) {
  if (!(y > 0.f) || !std::isfinite(y)) return false;
  const float z = (float)(1.0 / (double)y);
  if (!std::isfinite(z) || !(z > 0.f) || !std::isnormal(z)) return false;
  for (int c = 0; c < 0x7E; ++c) {
    const double mid = 0.5 * (e4m3_positive(c) + e4m3_positive(c + 1));   // a boundary
    const double lo = mid * (1.0 - std::ldexp(1.0, -20)) * y;
    const double hi = mid * (1.0 + std::ldexp(1.0, -20)) * y;
    if (lo > 1.0) break;   // no p in (0, 1] reaches this boundary
    float p = std::nextafter((float)lo, 0.f);
    const float end = std::nextafter((float)std::min(hi, 1.0), 2.f);
    for (; p <= end && p <= 1.f; p = std::nextafter(p, 2.f)) {
      if (!std::isnormal(p)) continue;
      if (fast_quotient(p, y, z) != exact_quotient(p, y)) return false;
    }
  }
  *z_out = z;
  return true;
}

}  // namespace

extern "C" {

const char* kvq_status_string(kvq_status s) {
  switch (s) {
    case KVQ_OK: return "ok";
    case KVQ_ERR_INVALID: return "invalid argument";
    case KVQ_ERR_UNSUPPORTED: return "unsupported configuration";
    case KVQ_ERR_WORKSPACE: return "workspace too small";
    case KVQ_ERR_CUDA: return "CUDA error";
    default: return "unknown status";
  }
}

kvq_status kvq_tensor_scale(int fmt, float amax, float* scale_out) {
  if (!scale_out) return KVQ_ERR_INVALID;
  if (!std::isfinite(amax) || amax < 0.f) return KVQ_ERR_INVALID;
  float top;
  if (fmt == KVQ_FP8_E4M3) top = 448.0f;
  else if (fmt == KVQ_NVFP4) top = 2688.0f;
  else return KVQ_ERR_INVALID;
  *scale_out = amax == 0.f ? 1.0f : amax / top;   // one IEEE fp32 division
  return KVQ_OK;
}

kvq_status kvq_amax_bf16(const void* x, size_t n, float* amax_out, void* stream) {
  if (!amax_out || (n > 0 && !x)) return KVQ_ERR_INVALID;
  return cuda_status(
      launch_amax_bf16(static_cast<const uint16_t*>(x), n, amax_out, as_stream(stream)));
}

kvq_status kvq_encode_e4m3(const float* x, uint8_t* out, size_t n, void* stream) {
  if (n > 0 && (!x || !out)) return KVQ_ERR_INVALID;
  return cuda_status(launch_encode(0, x, out, n, as_stream(stream)));
}

kvq_status kvq_encode_e2m1(const float* x, uint8_t* out, size_t n, void* stream) {
  if (n > 0 && (!x || !out)) return KVQ_ERR_INVALID;
  return cuda_status(launch_encode(1, x, out, n, as_stream(stream)));
}

kvq_status kvq_quantize_fp8(const void* x, size_t n, float scale, const float* head_scale,
                            int head_len, int num_heads, uint8_t* out, void* stream) {
  if (n == 0) return KVQ_OK;
  if (!x || !out || !aligned16(x) || n % 8 != 0) return KVQ_ERR_INVALID;
  if (head_scale) {
    if (head_len <= 0 || head_len % 8 != 0 || num_heads <= 0) return KVQ_ERR_INVALID;
  } else if (!finite_pos(scale)) {
    return KVQ_ERR_INVALID;
  }
  const float z = head_scale ? 0.f : (float)(1.0 / (double)scale);
  return cuda_status(launch_quantize_fp8(static_cast<const uint16_t*>(x), n, scale, z, head_scale,
                                         head_len, num_heads, out, as_stream(stream)));
}

kvq_status kvq_encode_prob_e4m3(const float* p, uint8_t* out, size_t n, float prob_scale,
                                int* used_reciprocal, void* stream) {
  if (!std::isfinite(prob_scale) || !(prob_scale > 0.f)) return KVQ_ERR_INVALID;
  if (n > 0 && (!p || !out)) return KVQ_ERR_INVALID;
  float z = 0.f;
  const int fast = prob_reciprocal_ok(prob_scale, &z) ? 1 : 0;
  if (used_reciprocal) *used_reciprocal = fast;
  return cuda_status(launch_encode_prob(p, out, n, prob_scale, z, fast, as_stream(stream)));
}

kvq_status kvq_quantize_append(const kvq_cache* c, const void* k_new, const void* v_new,
                               const void* kpe_new, const int32_t* start_pos, int batch,
                               int n_tokens, void* stream) {
  kvq_status s = check_cache(c);
  if (s != KVQ_OK) return s;
  if (batch < 0 || n_tokens < 0) return KVQ_ERR_INVALID;
  if (batch == 0 || n_tokens == 0) return KVQ_OK;
  if (!k_new || !aligned16(k_new) || !start_pos) return KVQ_ERR_INVALID;
  if (c->fmt == KVQ_FP8_E4M3 && c->head_dim % 8 != 0) return KVQ_ERR_INVALID;
  if (is_mla(c)) {
    if (v_new || !kpe_new || !aligned16(kpe_new)) return KVQ_ERR_INVALID;
  } else {
    if (!v_new || !aligned16(v_new) || kpe_new) return KVQ_ERR_INVALID;
  }
  if ((long long)batch * n_tokens * c->num_kv_heads * c->head_dim >= (1LL << 40))
    return KVQ_ERR_UNSUPPORTED;
  if (batch > 32767 || c->num_kv_heads > 65535 || n_tokens >= (1 << 30))
    return KVQ_ERR_UNSUPPORTED;
  AppendArgs a{};
  a.fmt = c->fmt;
  a.D = c->head_dim;
  a.Hkv = c->num_kv_heads;
  a.ps = c->page_size;
  a.max_pages = c->max_pages_per_seq;
  a.num_pages = c->num_pages;
  a.batch = batch;
  a.T = n_tokens;
  a.rope = is_mla(c) ? c->rope_dim : 0;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.kpe_new = static_cast<const uint16_t*>(kpe_new);
  a.start_pos = start_pos;
  a.block_table = c->block_table;
  a.k_codes = static_cast<uint8_t*>(c->k_codes);
  a.v_codes = static_cast<uint8_t*>(c->v_codes);
  a.k_bscale = static_cast<uint8_t*>(c->k_bscale);
  a.v_bscale = static_cast<uint8_t*>(c->v_bscale);
  a.k_pe = static_cast<uint16_t*>(c->k_pe);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  // RN(1/scale): the double quotient rounded to fp32 is the correctly rounded
  // fp32 reciprocal (53 >= 2 * 24 + 2)
  a.k_recip = (float)(1.0 / (double)c->k_scale);
  a.v_recip = is_mla(c) ? a.k_recip : (float)(1.0 / (double)c->v_scale);
  a.k_hs = c->k_head_scale;
  a.v_hs = c->v_head_scale;
  a.has_v = is_mla(c) ? 0 : 1;
  return cuda_status(launch_append(a, as_stream(stream)));
}

kvq_status kvq_norm_rope(const kvq_rotary* r, int head_dim, int num_tokens,
                         const int32_t* positions, const kvq_heads* q, const kvq_heads* q_out,
                         int q_fp8, float q_scale, const float* q_head_scale, const kvq_heads* k,
                         const kvq_heads* k_out, int32_t* error_flag, void* stream) {
  if (head_dim < 1 || num_tokens < 0) return KVQ_ERR_INVALID;
  kvq_status s = check_rotary(r, head_dim);
  if (s != KVQ_OK) return s;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  if (!q && !k) return KVQ_ERR_INVALID;
  if (num_tokens == 0) return KVQ_OK;
  if (q) {
    s = check_query_rows(q, q_out, head_dim, num_tokens, q_fp8, q_scale, q_head_scale);
    if (s != KVQ_OK) return s;
  }
  if (k) {
    s = check_heads(k, head_dim, num_tokens, false);
    if (s == KVQ_OK) s = check_heads(k_out, head_dim, num_tokens, true);
    if (s != KVQ_OK) return s;
    if (k_out->num_heads != k->num_heads) return KVQ_ERR_INVALID;
  }
  if (r->rot_dim > 0 && !positions) return KVQ_ERR_INVALID;
  const long long heads = (q ? (long long)q->num_heads : 0) + (k ? (long long)k->num_heads : 0);
  if (num_tokens * heads >= (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  RopeArgs a{};
  rotary_args(a, r);
  a.q = rope_rows(q);
  a.k = rope_rows(k);
  a.q_out = rope_rows(q ? q_out : nullptr);
  a.k_out = rope_rows(k ? k_out : nullptr);
  a.q_norm = q ? r->q_norm : nullptr;
  a.k_norm = k ? r->k_norm : nullptr;
  a.tokens = (unsigned)num_tokens;
  a.positions = positions;
  a.q_fp8 = q ? q_fp8 : 0;
  a.q_scale = q_scale;
  a.q_recip = a.q_fp8 && !q_head_scale ? (float)(1.0 / (double)q_scale) : 0.f;
  a.q_hs = q_head_scale;
  a.error_flag = error_flag;
  return cuda_status(launch_rope(head_dim, false, a, as_stream(stream)));
}

kvq_status kvq_rope_append(const kvq_cache* c, const kvq_rotary* r, int batch, int n_tokens,
                           const int32_t* start_pos, const int32_t* new_lens, const kvq_heads* k,
                           const kvq_heads* v, const kvq_heads* kpe, const kvq_heads* q,
                           const kvq_heads* q_out, int q_fp8, float q_scale,
                           const float* q_head_scale, int32_t* error_flag, void* stream) {
  RopeArgs where{};
  where.start_pos = start_pos;
  where.new_lens = new_lens;
  where.T = n_tokens;
  const long long tokens = batch < 0 || n_tokens < 0 ? -1 : (long long)batch * n_tokens;
  return rope_append(c, r, tokens, k, v, kpe, q, q_out, q_fp8, q_scale,
                     q_head_scale, error_flag, where, as_stream(stream));
}

kvq_status kvq_rope_append_slots(const kvq_cache* c, const kvq_rotary* r, int num_tokens,
                                 const int32_t* positions, const int64_t* slots,
                                 const kvq_heads* k, const kvq_heads* v, const kvq_heads* kpe,
                                 const kvq_heads* q, const kvq_heads* q_out, int q_fp8,
                                 float q_scale, const float* q_head_scale, int32_t* error_flag,
                                 void* stream) {
  RopeArgs where{};
  where.positions = positions;
  where.slots = reinterpret_cast<const long*>(slots);
  return rope_append(c, r, num_tokens, k, v, kpe, q, q_out, q_fp8, q_scale, q_head_scale,
                     error_flag, where, as_stream(stream));
}

kvq_status kvq_plan_step(const kvq_page_plan* p, void* stream) {
  if (!p || p->batch < 0 || p->page_size < 1 || p->num_pages < 1 || p->max_pages_per_seq < 1 ||
      p->max_tokens < 0)
    return KVQ_ERR_INVALID;
  if (!p->free_pages || !p->free_count || !p->free_count_out || !p->counter) return KVQ_ERR_INVALID;
  if (p->batch > 0 && (!p->block_table || !p->seq_lens || !p->seq_lens_out || !p->add_lens))
    return KVQ_ERR_INVALID;
  if (p->batch > kMaxPlanBatch || p->max_tokens > (1 << 30) || p->num_pages > (1 << 30) ||
      (long long)p->max_pages_per_seq * p->page_size >= (1LL << 31))
    return KVQ_ERR_UNSUPPORTED;
  PlanArgs a{};
  a.batch = p->batch;
  a.ps = p->page_size;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages_per_seq;
  a.max_tokens = p->max_tokens;
  divisor(p->page_size, &a.ps_mul, &a.ps_shift);
  a.block_table = p->block_table;
  a.seq_lens = p->seq_lens;
  a.seq_lens_out = p->seq_lens_out;
  a.add_lens = p->add_lens;
  a.free_pages = p->free_pages;
  a.free_count = p->free_count;
  a.free_count_out = p->free_count_out;
  a.counter = p->counter;
  a.start_pos = p->start_pos;
  a.q_offsets = p->q_offsets;
  a.slots = reinterpret_cast<long*>(p->slots);
  a.positions = p->positions;
  a.error_flag = p->error_flag;
  return cuda_status(launch_plan(a, as_stream(stream)));
}

kvq_status kvq_auto_splits(int num_sms, int batch, int num_kv_heads, int q_per_kv,
                           int max_kv_len, int fmt, int* out_s) {
  if (!out_s || num_sms < 1 || batch < 1 || num_kv_heads < 1 || max_kv_len < 0)
    return KVQ_ERR_INVALID;
  // When the (request, kv head) groups fit in one wave of the partial kernel
  // (two resident six-warp CTAs per SM, or three four-warp CTAs without wide
  // CTAs; two with more than eight query heads per kv head; one for the MLA
  // kernel: NVFP4, one kv head, 16 query heads), s fills that wave: a partly
  // filled second wave costs more than idle slots in the first (GQA FP8 batch
  // 16 x 8 kv heads at 8192 tokens: 52.3 us at s = 2, one wave, against 57.3
  // at s = 4 and 69.3 at s = 3; batch 8 at 32768: 91.6 us at s = 4 against
  // 106.6 at s = 16 and 128.7 at s = 5).  When they do not, the grid runs in
  // several waves anyway and chunks of at most kTargetChunk tokens cut long
  // or ragged requests into pieces that balance across them.
  // More than kManySplits splits of chunks shorter than kShortChunk tokens
  // lose to fewer, longer chunks (per-CTA fixed cost; the fused merge stages
  // about 30 splits in shared memory): measured on 8 kv-head groups at 8192
  // tokens, 28 splits 18.5 us against 21.0 us at 57.
  constexpr long long kMinChunk = 128, kMaxSplits = 64, kTargetChunk = 2048;
  constexpr long long kShortChunk = 256, kManySplits = 32;
  const bool mla_shape = fmt == KVQ_NVFP4 && num_kv_heads == 1 && q_per_kv == 16;
  const long long ctas_per_sm = mla_shape ? 1 : q_per_kv > 8 ? 2 : kWideCta ? 2 : 3;
  const long long base = (long long)batch * num_kv_heads;
  long long s = ctas_per_sm * num_sms / base;
  if (s < 1) s = ((long long)max_kv_len + kTargetChunk - 1) / kTargetChunk;
  if (s > kManySplits && (long long)max_kv_len < s * kShortChunk)
    s = std::max(kManySplits, ((long long)max_kv_len + kShortChunk - 1) / kShortChunk);
  const long long by_len = max_kv_len / kMinChunk;
  if (s > by_len) s = by_len;
  if (s < 1) s = 1;
  if (s > kMaxSplits) s = kMaxSplits;
  *out_s = (int)s;
  return KVQ_OK;
}

kvq_status kvq_shared_splits(int num_sms, int batch, int num_kv_heads, int q_per_kv,
                             int prefix_len, int max_own_len, int fmt, int* prefix_splits,
                             int* own_splits) {
  if (!prefix_splits || !own_splits || prefix_len < 0 || max_own_len < 0 || q_per_kv < 1)
    return KVQ_ERR_INVALID;
  if (num_sms < 1 || batch < 1 || num_kv_heads < 1 ||
      (fmt != KVQ_FP8_E4M3 && fmt != KVQ_NVFP4))
    return KVQ_ERR_INVALID;
  // A model of the step in microseconds, from measurements on GB300 (FP8,
  // head_dim 128, probabilities in two parts; other formats, head dims and one
  // part are taken for the same): the prefix's kernel runs one CTA per SM, kTile
  // per token tile and kFixed around them (256-row tiles; 128-row ones kTile1, kFixed1);
  // the requests' own chunks take kOwn + kOwnToken per token (half the longest
  // is taken as the mean), two CTAs on each SM that the prefix leaves free,
  // and the rest when it is done.  Merging adds kMerge per partial of a row
  // (where own chunks merge in place, more with the q_per_kv rows that a CTA
  // merges, from four on: 96 requests x 8k with 16 rows each, probabilities in one
  // part, take 31.2 us with 16 splits merged in place, 27.0 with 18 and the merging
  // launch), and a launch of its own kMergeLaunch where not all own chunks fit
  // beside the prefix.
  constexpr double kTile = 2.2, kFixed = 6, kTile1 = 1.5, kFixed1 = 5.5;
  constexpr double kOwn = 5, kOwnToken = 0.01, kMerge = 0.12, kMergeLaunch = 4;
  const bool wide = (long long)batch * q_per_kv > 128;
  const long long base = num_kv_heads * shared_row_tiles(batch, q_per_kv);
  const long long groups = (long long)batch * num_kv_heads;
  const long long tiles = ((long long)prefix_len + 127) / 128;
  double best = 0;
  *prefix_splits = *own_splits = 0;
  for (int so = 1; so <= 16; so *= 2) {
    if (so > 1 && max_own_len < 128 * so) break;   // at least 128 tokens per chunk
    const double own = groups * so;
    const double t_own = kOwn + kOwnToken * 0.5 * max_own_len / so;
    for (int sp = 1; sp <= std::max<long long>(1, std::min<long long>(tiles, 64 - so)); ++sp) {
      const long long ctas = base * sp;
      const double waves = (double)((ctas + num_sms - 1) / num_sms);
      const double t_prefix = waves * ((double)((tiles + sp - 1) / sp) * (wide ? kTile : kTile1) +
                                       (wide ? kFixed : kFixed1));
      const double room = 2.0 * (double)std::max<long long>(0, num_sms - ctas);
      double t = t_prefix + kMerge * (sp + so);
      if (own <= room) {
        t = std::max(t_prefix, t_own) + kMerge * std::max(1.0, q_per_kv / 4.0) * (sp + so);
      } else {
        const double beside = room * std::floor(t_prefix / t_own);
        t += kMergeLaunch;
        if (own > beside) t += std::ceil((own - beside) / (2.0 * num_sms)) * t_own;
      }
      if (*prefix_splits == 0 || t < best) {
        best = t;
        *prefix_splits = sp;
        *own_splits = so;
      }
    }
  }
  return KVQ_OK;
}

size_t kvq_partial_workspace_bytes(int batch, int num_q_heads, int num_splits, int v_dim) {
  if (batch < 0 || num_q_heads < 0 || num_splits < 0 || v_dim < 0) return 0;
  const size_t rows = (size_t)batch * num_q_heads * num_splits;
  return rows * (size_t)v_dim * sizeof(float) + rows * sizeof(float);
}

}  // extern "C"

namespace {

// Shared body of kvq_decode_partial and kvq_decode (fused when counters), and
// of kvq_decode_shared: with prefix_splits > 0 the requests start at token
// prefix_len, and the merge takes the preceding kernel's prefix_splits partials
// in too.  Of kvq_decode_diff: with `diff`, each query head is two rows.  And of
// kvq_chunk_attention: with q_offsets, for the requests that have one of num_tokens rows.
kvq_status decode_impl(const kvq_cache* c, const kvq_decode_params* p, const void* q,
                       float* part_o, float* part_lse, uint32_t* counters, void* out,
                       cudaStream_t stream, int prefix_len = 0, int prefix_splits = 0,
                       uint32_t* ready = nullptr, const kvq_diff* diff = nullptr,
                       const int32_t* q_offsets = nullptr, int num_tokens = 0,
                       const int32_t* longest = nullptr) {
  kvq_status s = check_cache(c);
  if (s != KVQ_OK) return s;
  s = check_params(p);
  if (s != KVQ_OK) return s;
  if (p->batch == 0) return KVQ_OK;
  if (!q || !aligned16(q) || !part_o || !aligned16(part_o) || !part_lse) return KVQ_ERR_INVALID;
  if (counters && !out) return KVQ_ERR_INVALID;
  if (counters && p->num_splits > kMaxFusedSplits) return KVQ_ERR_UNSUPPORTED;
  if (p->num_q_heads % c->num_kv_heads != 0) return KVQ_ERR_INVALID;
  const int maps = diff ? 2 : 1;
  if (p->num_q_heads / c->num_kv_heads > kMaxGroup / maps) return KVQ_ERR_UNSUPPORTED;
  const int G = maps * (p->num_q_heads / c->num_kv_heads);
  if ((long long)p->max_kv_len > (long long)c->max_pages_per_seq * c->page_size)
    return KVQ_ERR_INVALID;
  if ((long long)p->batch * c->num_kv_heads >= (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  const bool probq = p->prob_scale > 0.f;
  long long score_floats = 0;
  if (probq) {
    long long chunk = ((long long)p->max_kv_len + p->num_splits - 1) / p->num_splits;
    chunk = (chunk + 15) / 16 * 16;
    score_floats = chunk * G;
    if (score_floats > kScoreCapacity) return KVQ_ERR_UNSUPPORTED;
  }
  const int D = c->head_dim;
  const uint64_t rows = (uint64_t)c->num_pages * c->num_kv_heads * c->page_size;

  PartialArgs a{};
  a.q = q;
  a.q_fp8 = p->q_fp8;
  a.q_scale = p->q_scale;
  a.q_hs = p->q_fp8 ? p->q_head_scale : nullptr;
  a.k_bscale = static_cast<const uint8_t*>(c->k_bscale);
  a.v_bscale = static_cast<const uint8_t*>(c->v_bscale);
  a.k_pe = static_cast<const uint16_t*>(c->k_pe);
  a.block_table = c->block_table;
  a.seq_lens = p->seq_lens;
  a.part_o = part_o;
  a.part_lse = part_lse;
  a.error_flag = p->error_flag;
  a.batch = p->batch;
  a.Hq = G * c->num_kv_heads;
  a.Hkv = c->num_kv_heads;
  a.G = G;
  a.ps = c->page_size;
  a.max_pages = c->max_pages_per_seq;
  a.num_pages = c->num_pages;
  a.num_splits = p->num_splits;
  a.part_splits = p->num_splits;
  a.max_kv_len = p->max_kv_len;
  a.Dv = p->v_dim;
  a.score_floats = (int)score_floats;
  a.qk_scale_log2 = p->sm_scale * c->k_scale * 1.4426950408889634f;
  a.sm_scale = p->sm_scale;
  a.k_hs = c->k_head_scale;
  a.v_hs = c->v_head_scale;
  a.prob_scale = p->prob_scale;
  if (probq) a.prob_fast = prob_reciprocal_ok(p->prob_scale, &a.prob_recip) ? 1 : 0;
  a.fresh = p->fresh_tokens;
  if (prefix_splits > 0) {
    a.fresh = 0;
    a.part_splits = p->num_splits + prefix_splits;
    a.skip = prefix_len;
    a.late_merge = 1;
    a.ready = ready;
  }
  a.counters = counters;
  a.out = out;
  a.out_dtype = p->out_dtype;
  a.out_scale = p->out_scale;

  if (is_mla(c)) {
    if (D != 512 || c->rope_dim != 64 || G != 16 || p->qk_dim != 576 || p->v_dim != 512)
      return KVQ_ERR_UNSUPPORTED;
    if (probq || p->q_fp8) return KVQ_ERR_UNSUPPORTED;
    a.out_mult = c->k_scale;   // the values are the latent itself
    a.pe_scale_log2 = p->sm_scale * 1.4426950408889634f;
    // latent codes as two 128-byte halves per row, rope keys as 128-byte rows,
    // both in 16-row boxes with the 128-byte swizzle
    // (and 64-row boxes for tiles inside one page)
    CUtensorMap tkv, tpe, tkv64, tpe64;
    if (!make_slice_map(&tkv, c->k_codes, 128, 2, rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_row_map(&tpe, c->k_pe, 128, rows) ||
        !make_slice_map(&tkv64, c->k_codes, 128, 2, rows, CU_TENSOR_MAP_SWIZZLE_128B,
                        rows >= 64 ? 64 : kBoxTokens) ||
        !make_row_map(&tpe64, c->k_pe, 128, rows, rows >= 64 ? 64 : kBoxTokens))
      return KVQ_ERR_CUDA;
    return cuda_status(launch_mla_partial(tkv, tpe, tkv64, tpe64, a, stream));
  }
  if (p->qk_dim != D || p->v_dim != D) return KVQ_ERR_INVALID;
  const bool ok_dims = (c->fmt == KVQ_FP8_E4M3 && (D == 64 || D == 128)) ||
                       (c->fmt == KVQ_NVFP4 && (D == 64 || D == 128 || D == 256));
  if (!ok_dims) return KVQ_ERR_UNSUPPORTED;
  a.out_mult = probq ? c->v_scale * p->prob_scale : c->v_scale;
  const uint64_t row_bytes = c->fmt == KVQ_FP8_E4M3 ? D : D / 2;
  TensorMaps m;
  if (!make_row_map(&m.k16, c->k_codes, row_bytes, rows) ||
      !make_row_map(&m.v16, c->v_codes, row_bytes, rows))
    return KVQ_ERR_CUDA;
  a.q_offsets = q_offsets;
  a.num_tokens = num_tokens;
  a.longest = longest;
  if (diff) {
    a.diff_lambda = diff->lambda;
    a.diff_norm = diff->norm;
    a.diff_eps = diff->eps;
    a.diff_gain = diff->gain;
    return cuda_status(launch_partial_diff(c->fmt, D, m, a, stream));
  }
  if (q_offsets) return cuda_status(launch_partial_packed(c->fmt, D, m, a, stream));
  return cuda_status(launch_partial(c->fmt, D, probq, m, a, stream));
}

}  // namespace

extern "C" {

kvq_status kvq_decode_partial(const kvq_cache* c, const kvq_decode_params* p, const void* q,
                              float* part_o, float* part_lse, void* stream) {
  return decode_impl(c, p, q, part_o, part_lse, nullptr, nullptr, as_stream(stream));
}

kvq_status kvq_decode(const kvq_cache* c, const kvq_decode_params* p, const void* q,
                      float* part_o, float* part_lse, uint32_t* counters, void* out,
                      void* stream) {
  if (p && p->batch > 0 && (!counters || !out)) return KVQ_ERR_INVALID;
  return decode_impl(c, p, q, part_o, part_lse, counters, out,
                     as_stream(stream));
}

kvq_status kvq_decode_diff(const kvq_cache* c, const kvq_decode_params* p, const kvq_diff* d,
                           const void* q, float* part_o, float* part_lse, uint32_t* counters,
                           void* out, void* stream) {
  kvq_status s = check_cache(c);
  if (s != KVQ_OK) return s;
  s = check_params(p);
  if (s == KVQ_OK) s = check_diff(d);
  if (s != KVQ_OK) return s;
  if (is_mla(c) || p->prob_scale > 0.f) return KVQ_ERR_UNSUPPORTED;
  s = check_heads_of(c, p, true);
  if (s != KVQ_OK) return s;
  if (p->num_q_heads / c->num_kv_heads > kMaxGroup / 2) return KVQ_ERR_UNSUPPORTED;
  if (p->batch > 0 && (!counters || !out)) return KVQ_ERR_INVALID;
  return decode_impl(c, p, q, part_o, part_lse, counters, out, as_stream(stream), 0, 0, nullptr, d);
}

kvq_status kvq_decode_shared(const kvq_cache* c, const kvq_decode_params* p, int prefix_len,
                             const int32_t* prefix_table, int prefix_splits, const void* q,
                             float* part_o, float* part_lse, uint32_t* counters, void* out,
                             void* stream) {
  kvq_status s = check_cache(c);
  if (s != KVQ_OK) return s;
  s = check_params(p);
  if (s != KVQ_OK) return s;
  if (prefix_len < 0 || prefix_len % c->page_size != 0 || prefix_len > p->max_kv_len)
    return KVQ_ERR_INVALID;
  if (prefix_len > 0 && prefix_splits < 1) return KVQ_ERR_INVALID;
  if (p->prefix_p_f16 != 0 && p->prefix_p_f16 != 1) return KVQ_ERR_INVALID;
  if (p->batch > 0 && (!q || !aligned16(q) || !part_o || !part_lse || !counters || !out))
    return KVQ_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(part_o) & 31u) return KVQ_ERR_INVALID;
  if (p->num_q_heads % c->num_kv_heads != 0) return KVQ_ERR_INVALID;
  if (is_mla(c) || p->prob_scale > 0.f) return KVQ_ERR_UNSUPPORTED;
  // token numbers are 32-bit, and each lane's (32 boxes of up to 128 tokens) is formed
  // before it is compared
  if (prefix_len > INT_MAX - 4096) return KVQ_ERR_UNSUPPORTED;
  const int D = c->head_dim;
  if (p->qk_dim != D || p->v_dim != D) return KVQ_ERR_INVALID;
  if (D != 64 && D != 128) return KVQ_ERR_UNSUPPORTED;
  const int G = p->num_q_heads / c->num_kv_heads;
  if (G > kMaxGroup) return KVQ_ERR_UNSUPPORTED;
  if ((long long)p->max_kv_len > (long long)c->max_pages_per_seq * c->page_size)
    return KVQ_ERR_INVALID;
  if (p->batch == 0) return KVQ_OK;
  if (prefix_len == 0)
    return decode_impl(c, p, q, part_o, part_lse, counters, out, as_stream(stream));
  // a prefix split holds at least one 128-token tile
  const int tiles = (prefix_len + 127) / 128;
  if (prefix_splits > tiles) prefix_splits = tiles;
  if (p->num_splits + prefix_splits > kMaxFusedSplits) return KVQ_ERR_UNSUPPORTED;
  if ((long long)p->batch * p->num_q_heads * (p->num_splits + prefix_splits) >= (1LL << 31) ||
      c->num_kv_heads > 65535)
    return KVQ_ERR_UNSUPPORTED;
  SharedArgs a{};
  a.q = q;
  a.q_fp8 = p->q_fp8;
  a.q_scale = p->q_scale;
  a.q_hs = p->q_fp8 ? p->q_head_scale : nullptr;
  a.k_bscale = static_cast<const uint8_t*>(c->k_bscale);
  a.v_bscale = static_cast<const uint8_t*>(c->v_bscale);
  a.prefix_table = prefix_table;
  a.block_table = c->block_table;
  a.batch = p->batch;
  a.max_pages = c->max_pages_per_seq;
  a.seq_lens = p->seq_lens;
  a.part_o = part_o;
  a.part_lse = part_lse;
  a.error_flag = p->error_flag;
  a.R = p->batch * G;
  a.G = G;
  a.Hq = p->num_q_heads;
  a.Hkv = c->num_kv_heads;
  a.ps = c->page_size;
  a.num_pages = c->num_pages;
  a.prefix = prefix_len;
  a.splits = prefix_splits;
  a.box = box_rows(c->page_size);
  a.wide_p = p->prefix_p_f16 == 0;
  a.sm_scale = p->sm_scale;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.k_hs = c->k_head_scale;
  a.v_hs = c->v_head_scale;
  a.ready = counters;
  a.ready_n = p->batch * c->num_kv_heads;   // < 2^31, as partials are
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KVQ_ERR_CUDA;
  const long long base = shared_row_tiles(p->batch, G) * c->num_kv_heads;
  a.split0 = p->num_splits;
  a.part_splits = p->num_splits + prefix_splits;
  // The requests' own chunks run beside the prefix on the SMs that it leaves
  // free.  If those hold all of them at once, each waits there for the prefix
  // and merges; otherwise they only write their partials, so that waiting ones
  // keep no others out, and a third launch merges.
  const long long free_ctas = 2 * (sms - base * prefix_splits);
  const bool fused = (long long)p->batch * c->num_kv_heads * p->num_splits <= free_ctas;
  const uint64_t rows = (uint64_t)c->num_pages * c->num_kv_heads * c->page_size;
  const uint64_t row_bytes = c->fmt == KVQ_FP8_E4M3 ? D : D / 2;
  TensorMaps maps;
  if (!make_row_map(&maps.k16, c->k_codes, row_bytes, rows, (uint32_t)a.box) ||
      !make_row_map(&maps.v16, c->v_codes, row_bytes, rows, (uint32_t)a.box))
    return KVQ_ERR_CUDA;
  s = cuda_status(launch_shared_prefix(c->fmt, D, maps, a, as_stream(stream)));
  if (s != KVQ_OK) return s;
  s = decode_impl(c, p, q, part_o, part_lse, fused ? counters : nullptr, out, as_stream(stream),
                  prefix_len, prefix_splits, counters);
  if (s != KVQ_OK || fused) return s;
  CombineArgs m{};
  m.part_o = part_o;
  m.part_lse = part_lse;
  m.out = out;
  m.rows = p->batch * p->num_q_heads;
  m.num_splits = a.part_splits;
  m.Dv = D;
  m.out_dtype = p->out_dtype;
  m.out_scale = p->out_scale;
  return cuda_status(launch_merge_rows(m, as_stream(stream)));
}

kvq_status kvq_decode_combine(const kvq_decode_params* p, const float* part_o,
                              const float* part_lse, void* out, void* stream) {
  kvq_status s = check_params(p);
  if (s != KVQ_OK) return s;
  if (p->batch == 0) return KVQ_OK;
  if (!part_o || !aligned16(part_o) || !part_lse || !out || p->v_dim % 4 != 0)
    return KVQ_ERR_INVALID;
  if ((long long)p->batch * p->num_q_heads >= (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  if (p->num_splits > kMaxFusedSplits) return KVQ_ERR_UNSUPPORTED;
  CombineArgs a{};
  a.part_o = part_o;
  a.part_lse = part_lse;
  a.out = out;
  a.rows = p->batch * p->num_q_heads;
  a.num_splits = p->num_splits;
  a.Dv = p->v_dim;
  a.out_dtype = p->out_dtype;
  a.out_scale = p->out_scale;
  return cuda_status(launch_combine(a, as_stream(stream)));
}

size_t kvq_chunk_workspace_bytes(int num_sms, const kvq_cache* c, const kvq_decode_params* p,
                                 const kvq_diff* d) {
  if (num_sms < 1 || !c || !p || c->num_kv_heads < 1 || c->head_dim < 1 || p->batch < 0 ||
      p->num_q_heads < 1 || p->max_kv_len < 0)
    return 0;
  return chunk_parts(num_sms, c, p, d).bytes;
}

kvq_status kvq_chunk_attention(const kvq_cache* c, const kvq_decode_params* p, const kvq_diff* d,
                               int num_tokens, const int32_t* q_offsets, const void* q,
                               void* workspace, size_t workspace_bytes, void* out, void* stream) {
  kvq_status s = check_cache(c);
  if (s != KVQ_OK) return s;
  s = check_params(p);
  if (s == KVQ_OK && d) s = check_diff(d);
  if (s != KVQ_OK) return s;
  if (num_tokens < 0 || (p->prefix_p_f16 != 0 && p->prefix_p_f16 != 1)) return KVQ_ERR_INVALID;
  if (is_mla(c) || p->prob_scale > 0.f) return KVQ_ERR_UNSUPPORTED;
  s = check_heads_of(c, p, false);
  if (s != KVQ_OK) return s;
  const int G = p->num_q_heads / c->num_kv_heads, D = c->head_dim;
  if ((long long)num_tokens * G >= (1LL << 30) || p->batch > kMaxPlanBatch ||
      p->max_kv_len > INT_MAX - 4096)
    return KVQ_ERR_UNSUPPORTED;
  if (p->batch == 0 || num_tokens == 0) return KVQ_OK;
  if (!q || !aligned16(q) || !q_offsets || !out || (reinterpret_cast<uintptr_t>(out) & 31u))
    return KVQ_ERR_INVALID;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 31u)) return KVQ_ERR_INVALID;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KVQ_ERR_CUDA;
  const ChunkParts parts = chunk_parts(sms, c, p, d);
  if (workspace_bytes < parts.bytes) return KVQ_ERR_WORKSPACE;
  ChunkArgs a{};
  a.q = q;
  a.q_fp8 = p->q_fp8;
  a.q_scale = p->q_scale;
  a.q_hs = p->q_fp8 ? p->q_head_scale : nullptr;
  a.k_bscale = static_cast<const uint8_t*>(c->k_bscale);
  a.v_bscale = static_cast<const uint8_t*>(c->v_bscale);
  a.block_table = c->block_table;
  a.seq_lens = p->seq_lens;
  a.q_offsets = q_offsets;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.out = out;
  a.error_flag = p->error_flag;
  a.batch = p->batch;
  a.num_tokens = num_tokens;
  a.G = G;
  a.Hq = p->num_q_heads;
  a.Hkv = c->num_kv_heads;
  a.D = D;
  a.ps = c->page_size;
  a.max_pages = c->max_pages_per_seq;
  a.num_pages = c->num_pages;
  a.max_kv_len = p->max_kv_len;
  divisor(G, &a.g_mul, &a.g_shift);
  a.box = box_rows(c->page_size);
  a.wide_p = p->prefix_p_f16 == 0;
  a.out_dtype = p->out_dtype;
  a.out_scale = p->out_scale;
  a.sm_scale = p->sm_scale;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.k_hs = c->k_head_scale;
  a.v_hs = c->v_head_scale;
  if (d) {
    a.diff_lambda = d->lambda;
    a.diff_norm = d->norm;
    a.diff_eps = d->eps;
    a.diff_gain = d->gain;
  }
  const uint64_t rows = (uint64_t)c->num_pages * c->num_kv_heads * c->page_size;
  const uint64_t row_bytes = c->fmt == KVQ_FP8_E4M3 ? D : D / 2;
  TensorMaps maps;
  if (!make_row_map(&maps.k16, c->k_codes, row_bytes, rows, (uint32_t)a.box) ||
      !make_row_map(&maps.v16, c->v_codes, row_bytes, rows, (uint32_t)a.box))
    return KVQ_ERR_CUDA;
  uint8_t* const w = a.workspace;
  if (parts.splits > 0) a.counters = reinterpret_cast<uint32_t*>(w + parts.counters);
  a.single_splits = parts.splits;
  s = cuda_status(launch_shares(c->fmt, a, sms, as_stream(stream)));
  if (s != KVQ_OK) return s;
  if (parts.splits > 0) {
    kvq_decode_params one = *p;
    one.num_splits = parts.splits;
    one.fresh_tokens = 0;
    s = decode_impl(c, &one, q, reinterpret_cast<float*>(w + parts.o),
                    reinterpret_cast<float*>(w + parts.lse), a.counters, out, as_stream(stream), 0,
                    0, nullptr, d, q_offsets, num_tokens,
                    reinterpret_cast<const int32_t*>(w) + kChunkLongest);
    if (s != KVQ_OK) return s;
  }
  return cuda_status(launch_chunk(c->fmt, D, maps, a, sms, as_stream(stream)));
}

kvq_status kvq_prefill(const kvq_cache* c, const kvq_decode_params* p, int q_len, const void* q,
                       void* out, void* stream) {
  kvq_status s = check_cache(c);
  if (s != KVQ_OK) return s;
  s = check_params(p);
  if (s != KVQ_OK) return s;
  if (q_len < 1) return KVQ_ERR_INVALID;
  if (p->batch == 0) return KVQ_OK;
  if (!q || !aligned16(q) || !out) return KVQ_ERR_INVALID;
  if (p->num_q_heads % c->num_kv_heads != 0) return KVQ_ERR_INVALID;
  if (is_mla(c) || p->prob_scale > 0.f || p->q_fp8) return KVQ_ERR_UNSUPPORTED;
  const int D = c->head_dim;
  if (p->qk_dim != D || p->v_dim != D) return KVQ_ERR_INVALID;
  if (D != 64 && D != 128) return KVQ_ERR_UNSUPPORTED;
  if ((long long)p->max_kv_len > (long long)c->max_pages_per_seq * c->page_size)
    return KVQ_ERR_INVALID;
  const int G = p->num_q_heads / c->num_kv_heads;
  if ((long long)q_len * G >= (1LL << 30) || (long long)p->batch * c->num_kv_heads > 65535)
    return KVQ_ERR_UNSUPPORTED;
  PartialArgs a{};
  a.q = q;
  a.k_bscale = static_cast<const uint8_t*>(c->k_bscale);
  a.v_bscale = static_cast<const uint8_t*>(c->v_bscale);
  a.block_table = c->block_table;
  a.seq_lens = p->seq_lens;
  a.error_flag = p->error_flag;
  a.batch = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = c->num_kv_heads;
  a.G = G;
  a.ps = c->page_size;
  a.max_pages = c->max_pages_per_seq;
  a.num_pages = c->num_pages;
  a.max_kv_len = p->max_kv_len;
  a.Dv = D;
  a.q_len = q_len;
  a.qk_scale_log2 = p->sm_scale * c->k_scale * 1.4426950408889634f;
  a.sm_scale = p->sm_scale;
  a.k_hs = c->k_head_scale;
  a.v_hs = c->v_head_scale;
  a.out_mult = c->v_scale;
  a.out = out;
  a.out_dtype = p->out_dtype;
  a.out_scale = p->out_scale;
  const uint64_t rows = (uint64_t)c->num_pages * c->num_kv_heads * c->page_size;
  const uint64_t row_bytes = c->fmt == KVQ_FP8_E4M3 ? D : D / 2;
  TensorMaps maps;
  if (!make_row_map(&maps.k16, c->k_codes, row_bytes, rows) ||
      !make_row_map(&maps.v16, c->v_codes, row_bytes, rows))
    return KVQ_ERR_CUDA;
  return cuda_status(launch_prefill(c->fmt, D, maps, a, as_stream(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free decode.
//
// Some callers cannot allocate device memory for the split partials: their
// device memory is owned by a host framework that hands out only the tensors
// it planned (a serving engine's fixed memory pool), or they run under a hard
// memory budget where an extra cudaMalloc is not allowed.  kvq_decode_noalloc
// serves them from one buffer the library itself carries: a file-scope device
// array of KVQ_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds
// until the process exits.  In host code the array's name is only a stand-in
// for the symbol, so the device's real address is looked up with
// cudaGetSymbolAddress (with that device current) on every call and passed
// to the kernel.
// ---------------------------------------------------------------------------

static __device__ __align__(256) unsigned char g_noalloc_scratch[KVQ_NOALLOC_SCRATCH_BYTES];

namespace {

// Device address of the scratch array on the current device.  Looked up on
// every call: after the first call on a device (which loads the module) it is
// a table lookup, and it stays right if the device's context is torn down
// and created again (the module, and so the array, may then move).
kvq_status noalloc_scratch(void** out) {
  void* ptr = nullptr;
  if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || !ptr) return KVQ_ERR_CUDA;
  *out = ptr;
  return KVQ_OK;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

extern "C" kvq_status kvq_decode_noalloc(const kvq_cache* c, const kvq_decode_params* p,
                                         const void* q, void* out, void* stream) {
  kvq_status st = check_cache(c);
  if (st != KVQ_OK) return st;
  st = check_params(p);
  if (st != KVQ_OK) return st;
  if (p->batch == 0) return KVQ_OK;
  if (!q || !out) return KVQ_ERR_INVALID;
  // scratch layout: [arrival counters][partial lse][partial o], 256-byte aligned
  const size_t rows = (size_t)p->batch * p->num_q_heads * p->num_splits;
  const size_t counter_bytes = up256((size_t)p->batch * c->num_kv_heads * sizeof(uint32_t));
  const size_t lse_bytes = up256(rows * sizeof(float));
  const size_t o_bytes = rows * (size_t)p->v_dim * sizeof(float);
  if (counter_bytes + lse_bytes + o_bytes > KVQ_NOALLOC_SCRATCH_BYTES) return KVQ_ERR_WORKSPACE;
  void* base = nullptr;
  st = noalloc_scratch(&base);
  if (st != KVQ_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(base);
  uint32_t* counters = reinterpret_cast<uint32_t*>(w);
  float* part_lse = reinterpret_cast<float*>(w + counter_bytes);
  float* part_o = reinterpret_cast<float*>(w + counter_bytes + lse_bytes);
  // the arrival counters must start at zero (a previous call leaves them
  // zero; clearing them here keeps the contract independent of history)
  if (cudaMemsetAsync(counters, 0, counter_bytes, as_stream(stream)) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return decode_impl(c, p, q, part_o, part_lse, counters, out, as_stream(stream));
}
