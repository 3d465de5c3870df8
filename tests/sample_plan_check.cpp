// Prints how many CTAs sample a row, and a CTA's share, for "rows vocab cap sms" on each line of stdin.
#include <cstdio>

#include "sample_plan.cuh"

int main() {
  long long rows;
  int vocab, cap, sms;
  while (scanf("%lld %d %d %d", &rows, &vocab, &cap, &sms) == 4) {
    const int c = ls::sample_cluster(rows, vocab, cap, sms);
    printf("%d %d\n", c, ls::sample_share(vocab, c));
  }
  return 0;
}
