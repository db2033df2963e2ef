// Prints the form of the microscaled product that each call read from standard
// input takes: "T N K f4 aligned sms" -> "tokens-a-tile ranks wide".
#include <cstdio>

#include "mx_plan.h"

int main() {
  int T, N, K, f4, aligned, sms;
  while (std::scanf("%d %d %d %d %d %d", &T, &N, &K, &f4, &aligned, &sms) == 6) {
    const strata::LinPlan p = strata::plan_linear(T, N, K, f4 != 0, sms);
    const bool wide = p.nt == 0 && strata::plan_wide(T, N, K, f4 != 0, aligned != 0, sms);
    std::printf("%d %d %d\n", p.nt, p.splits, (int)wide);
  }
  return 0;
}
