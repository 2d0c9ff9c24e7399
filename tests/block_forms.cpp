// Prints the form (rows, columns and wavefronts of a workgroup, stages held, and whether its grid fits) that
// each 8-bit product on the standard input takes: lines of dx (0 or 1), rows, groups, tables (0 or 1), h_in,
// h_out.  Built and run by tests/test_block_forms.py.
#include <cstdio>

#include "../adapter_gemv_amd/csrc/sgmv_fp8_rules.h"

int main() {
  int dx, n, groups, grouped, h_in, h_out;
  while (std::scanf("%d %d %d %d %d %d", &dx, &n, &groups, &grouped, &h_in, &h_out) == 6) {
    const sgmv_host::BlockLaunch L = sgmv_host::fp8_launch(dx != 0, n, groups, grouped != 0, h_in, h_out);
    std::printf("%d %d %d %d %d\n", L.rows, L.cols, L.waves, L.buffers, L.fits() ? 1 : 0);
  }
  return 0;
}
