// Reads lines "lora|lora_grad T N K R L" and prints how the library divides the call:
// lora: tile tiles splits k_share ranges n_share; lora_grad: tiles splits n_share chunk chunks
// shares dx_cols k_cols.
#include <stdio.h>
#include <string.h>

#include "../../weight_only_bit_rtn_amd/csrc/lora_division.h"

int main() {
  char op[32];
  long long T, N, K, R, L;
  while (scanf("%31s %lld %lld %lld %lld %lld", op, &T, &N, &K, &R, &L) == 6) {
    const lowbit::LoraSizes s = {T, N, K, R, L};
    if (strcmp(op, "lora") == 0) {
      const lowbit::LoraDivision d = lowbit::divide_lora(s);
      printf("%d %lld %d %d %d %d\n", d.tile, (long long)d.tiles, d.splits, d.k_share, d.ranges, d.n_share);
    } else {
      const lowbit::LoraGradDivision d = lowbit::divide_lora_grad(s);
      printf("%lld %d %d %d %lld %lld %d %d\n", (long long)d.tiles, d.splits, d.n_share, d.chunk,
             (long long)d.chunks, (long long)d.shares, d.dx_cols, d.k_cols);
    }
  }
  return 0;
}
