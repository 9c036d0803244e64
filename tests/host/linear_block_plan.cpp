// Prints the kernel (fp8mot::LinearTile) that linear_block_plan takes for each
// "M N K" line of the standard input.
#include <cstdio>

#include "../../mlp_fp8_quant_amd/csrc/linear_block_plan.h"

int main() {
  using namespace fp8mot;
  long long m, n, k;
  while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
    const char* name = "?";
    switch (linear_block_plan(m, n, k)) {
      case kRows1x1: name = "rows 1x1"; break;
      case kRows1x2: name = "rows 1x2"; break;
      case kRows1x4: name = "rows 1x4"; break;
      case kRows2x1: name = "rows 2x1"; break;
      case kRows2x2: name = "rows 2x2"; break;
      case kRows2x4: name = "rows 2x4"; break;
      case kRows4x2: name = "rows 4x2"; break;
      case kRows4x4: name = "rows 4x4"; break;
      case kRows4x4Pair: name = "rows 4x4 pair"; break;
      case kTile256x128: name = "256x128"; break;
      case kTile128x128: name = "128x128"; break;
      case kTile128x128K2: name = "128x128 K2"; break;
      case kTile128x64K2: name = "128x64 K2"; break;
      case kTile128x64: name = "128x64"; break;
    }
    std::puts(name);
  }
  return 0;
}
