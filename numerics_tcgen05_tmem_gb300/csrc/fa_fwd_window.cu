// Entry point of the attention forward with a sliding window and sinks (BF16).
//
// Query i sees the keys j <= i with i - j < window, and the first `sinks` keys:
//   O_i = sum_j P_ij V_j,  P_ij = exp(scale S_ij - lse_i) over the visible j.
// It is the kernel of fa_fwd_kernel.cuh with its walk over the key blocks cut to those that some
// row of the CTA sees (KeyWalk), so the work grows with N * (window + sinks) instead of N^2, and
// with the window's edge masked like the diagonal.  A row whose first visited block is hidden
// from it keeps the shift -inf until a visible key arrives.  Kernels of its own (kWin) leave the
// unwindowed ones as they are: the mask costs registers and instructions in every block.
#include "fa_fwd_kernel.cuh"

extern "C" int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
                             int d, int window, int sinks, float scale, int stable, float beta,
                             const fa_row_stats* stats, void* stream) {
  fa::NvtxRange nvtx_range("fa_fwd_window");
  using namespace fa;
  clear_error();
  fwd::Params p;
  bool want_stats;
  int rc = check_window(window, sinks);
  if (rc || (rc = prepare_fwd(p, want_stats, q, k, v, o, lse, B, H, N, d, 1, scale, stable, beta, stats))) return rc;
  p.window = window < N ? window : N;
  p.sinks = sinks < N ? sinks : N;
  CUtensorMap tq, tk, tv;
  if ((rc = make_tmap_bhnd(&tq, q, B * H, N, d, fwd::kBlockM)) || (rc = make_tmap_bhnd(&tk, k, B * H, N, d, fwd::kBlockN)) ||
      (rc = make_tmap_bhnd(&tv, v, B * H, N, d, fwd::kBlockN)))
    return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? dispatch_fwd<64, false, true>(stable, want_stats, tq, tk, tv, p, s)
                 : dispatch_fwd<128, false, true>(stable, want_stats, tq, tk, tv, p, s);
}
