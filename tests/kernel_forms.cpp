// Prints the form (rows, columns and wavefronts of a workgroup) that each product on the standard
// input takes: lines of mode, rows, groups, tables (0 or 1), h_in, h_out.  Built and run by
// tests/test_kernel_forms.py.
#include <cstdio>

#include "../adapter_gemv_amd/csrc/sgmv_rules.h"

int main() {
  int mode, n, groups, grouped, h_in, h_out;
  while (std::scanf("%d %d %d %d %d %d", &mode, &n, &groups, &grouped, &h_in, &h_out) == 6) {
    const sgmv_host::Launch L = mode == sgmv_dev::kDw
                                    ? sgmv_host::dw_launch(groups, h_in, h_out)
                                    : sgmv_host::rows_launch(static_cast<sgmv_dev::Mode>(mode), n, groups,
                                                             grouped != 0, h_in, h_out);
    std::printf("%d %d %d %d\n", L.rows, L.cols, L.waves, L.fits() ? 1 : 0);
  }
  return 0;
}
