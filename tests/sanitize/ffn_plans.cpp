// Which tiles and how many parts of k the gated feed-forward's products get:
// the rules of gated_ffn.hip, host code, asked without a device.  Sizes
// "rows dim hidden dtype" on standard input; a line of numbers for each: tile
// and parts of the forward, of dx and of both weights' gradients by themselves,
// whether those are one launch, and their tiles and parts there (0 if not).
#include <cstdio>

#include "../../selective_state_space_vjp_amd/csrc/gated_ffn.hip"

using namespace ssmvjp;

int main() {
  long long rows, dim, hidden;
  int dtype;
  while (std::scanf("%lld %lld %lld %d", &rows, &dim, &hidden, &dtype) == 4) {
    const ssmvjp_ffn_desc d{rows, dim, hidden, SSMVJP_ACT_SILU, dtype};
    const size_t elem = dtype == SSMVJP_BF16 ? 2 : 4;
    const int parts = grads_parts(d);
    const GemmPlan f = gemm_plan(shape_of(rows, hidden, dim, 1, 1, true, true, elem));
    const Shape x = shape_of(rows, dim, hidden, 2 * parts, 1, false, true, elem), w = shape_of(hidden, dim, rows, parts, 2, false, false, elem);
    const GemmPlan ax = gemm_plan(x), aw = gemm_plan(w);
    GemmPlan px, pw;
    const bool one = grads_plan(x, w, px, pw);
    if (!one) px = pw = {0, 0};
    std::printf("%d %d %d %d %d %d %d %d %d %d %d\n", f.tile, f.split, ax.tile, ax.split, aw.tile, aw.split, (int)one, px.tile, px.split,
                pw.tile, pw.split);
  }
  return 0;
}
