// Split-KV decode of a packed step's single tokens: instantiations of the partial kernel's
// mode 2 (sm_103a).  The kernel is in kvq_decode.cuh, the merge in kvq_attn.cuh.

#include "kvq_decode.cuh"

namespace kvq {
using namespace decode_impl;
namespace {

template <int FMT, int D, bool QF8>
cudaError_t by_rows(const TensorMaps& m, const PartialArgs& a, cudaStream_t st) {
  if (a.G > 8) return launch_partial_t<FMT, D, false, 2, QF8, kDecodeWarps, false, 2>(m, a, st);
  constexpr int NW = D <= 128 && kWideCta ? kWideWarps : kDecodeWarps;   // (wide_cta)
  return launch_partial_t<FMT, D, false, 1, QF8, NW, false, 2>(m, a, st);
}

template <int FMT, int D>
cudaError_t by_query(const TensorMaps& m, const PartialArgs& a, cudaStream_t st) {
  return a.q_fp8 ? by_rows<FMT, D, true>(m, a, st) : by_rows<FMT, D, false>(m, a, st);
}

}  // namespace

cudaError_t launch_partial_packed(int fmt, int D, const TensorMaps& m, const PartialArgs& a,
                                  cudaStream_t st) {
  if (fmt == kFmtFp8 && D == 128) return by_query<kFmtFp8, 128>(m, a, st);
  if (fmt == kFmtFp8 && D == 64) return by_query<kFmtFp8, 64>(m, a, st);
  if (fmt == kFmtNvfp4 && D == 128) return by_query<kFmtNvfp4, 128>(m, a, st);
  if (fmt == kFmtNvfp4 && D == 64) return by_query<kFmtNvfp4, 64>(m, a, st);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
