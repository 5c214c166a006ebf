// Reads lines "linear|gated|linear_grad|gated_grad T N K" and prints for each the
// kernel and tile plan that the library takes on a device of argv[1] CUs, and the
// bytes of the shares' sums.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../weight_only_bit_rtn_amd/csrc/w8a8_plan.h"

using namespace lowbit;

static void print(int mt, int nt, const TilePlan& p, size_t bytes) {
  printf("%dx%d %s %zu\n", mt, nt, !p.rest ? "whole" : p.whole ? "both" : "shared", bytes);
}

int main(int argc, char** argv) {
  const int cus = argc > 1 ? atoi(argv[1]) : 256;
  char op[32];
  long long T, N, K;
  while (scanf("%31s %lld %lld %lld", op, &T, &N, &K) == 4) {
    const bool gated = strncmp(op, "gated", 5) == 0;
    if (strstr(op, "grad")) {
      const int steps = (int)((N + kStepN - 1) / kStepN) * (gated ? 2 : 1);
      const GradPlan p = grad_plan(T, K, steps, cus);
      print(kGradShapes[p.shape].mt, kGradShapes[p.shape].kt, p.tiles, p.part_bytes());
    } else if (few_takes(T, K, gated)) {
      printf("few%lld %s 0\n", T == 3 ? 4 : T, T * K <= kFusedMost ? "fused" : "codes");
    } else {
      const GemmPlan p = gemm_plan(T, N, K, gated, cus);
      if (p.shape < 0)
        printf("ring%lld whole 0\n", (T + 15) / 16);
      else
        print(kProductShapes[p.shape].mt, kProductShapes[p.shape].nt, p.tiles, p.part_bytes());
    }
  }
  return 0;
}
