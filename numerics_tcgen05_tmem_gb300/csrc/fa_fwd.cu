// Entry points of the attention forward over whole rows: BF16 (fa_fwd) and E4M3 (fa_fwd_fp8).
// The kernel, its method and its launch rules are in fa_fwd_kernel.cuh.
#include "fa_fwd_kernel.cuh"

extern "C" int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                      int causal, float scale, int stable, float beta, const fa_row_stats* stats, void* stream) {
  fa::NvtxRange nvtx_range("fa_fwd");
  using namespace fa;
  clear_error();
  fwd::Params p;
  bool want_stats;
  int rc = prepare_fwd(p, want_stats, q, k, v, o, lse, B, H, N, d, causal, scale, stable, beta, stats);
  if (rc) return rc;
  CUtensorMap tq, tk, tv;
  if ((rc = make_tmap_bhnd(&tq, q, B * H, N, d, fwd::kBlockM)) || (rc = make_tmap_bhnd(&tk, k, B * H, N, d, fwd::kBlockN)) ||
      (rc = make_tmap_bhnd(&tv, v, B * H, N, d, fwd::kBlockN)))
    return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? dispatch_fwd<64, false>(stable, want_stats, tq, tk, tv, p, s)
                 : dispatch_fwd<128, false>(stable, want_stats, tq, tk, tv, p, s);
}

extern "C" int fa_fwd_fp8(const void* q8, const void* k8, const void* v8, const float* descale, void* o, float* lse,
                          int B, int H, int N, int d, int causal, float scale, int stable, float beta,
                          const fa_row_stats* stats, void* stream) {
  fa::NvtxRange nvtx_range("fa_fwd_fp8");
  using namespace fa;
  clear_error();
  if (d != 64 && d != 128) return set_error(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (!descale) return set_error(FA_ERR_INVALID_ARG, "descale is NULL");
  if (reinterpret_cast<uintptr_t>(descale) & 3) return set_error(FA_ERR_INVALID_ARG, "descale is not 4-byte aligned");
  fwd::Params p;
  bool want_stats;
  int rc = prepare_fwd(p, want_stats, q8, k8, v8, o, lse, B, H, N, d, causal, scale, stable, beta, stats);
  if (rc) return rc;
  p.descale = descale;
  CUtensorMap tq, tk, tv;
  if ((rc = make_tmap_u8_bhnd(&tq, q8, B * H, N, d, fwd::kBlockM)) ||
      (rc = make_tmap_u8_bhnd(&tk, k8, B * H, N, d, fwd::kBlockN)) ||
      (rc = make_tmap_u8_bhnd(&tv, v8, B * H, N, d, fwd::kBlockN)))
    return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? dispatch_fwd<64, true>(stable, want_stats, tq, tk, tv, p, s)
                 : dispatch_fwd<128, true>(stable, want_stats, tq, tk, tv, p, s);
}
