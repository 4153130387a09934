// Reads "tokens rows cols" lines and prints the kernel that the 8-bit product takes for each.
#include <cstdio>

#include "int8_plan.h"

int main() {
  const char* names[] = {"256x256", "256x128", "128x64", "64x128", "64x64", "32x32", "32x16"};
  long long tokens, rows, cols;
  while (std::scanf("%lld %lld %lld", &tokens, &rows, &cols) == 3)
    std::puts(gptq::int8_by_rows(rows, tokens) ? "rows" : names[(int)gptq::int8_best(rows, cols, tokens).form]);
}
