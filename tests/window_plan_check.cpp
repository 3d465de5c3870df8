// attended_most against its definition: the largest attended_len of the lengths up to L.
#include <cstdio>
#include <initializer_list>

#include "ls_plan.cuh"

int main() {
  for (int window : {0, 1, 2, 64, 127, 128, 129, 130, 255, 256, 300, 512, 1000, 2147483647}) {
    ls::Plan p{};
    p.window = window;
    int most = 0;
    for (int L = 0; L <= 3000; ++L) {
      const int here = ls::attended_len(p, L);
      if (here > most) most = here;
      if (ls::attended_most(p, L) != most) {
        printf("window %d, length %d: %d, not %d\n", window, L, ls::attended_most(p, L), most);
        return 1;
      }
    }
  }
  printf("ok\n");
  return 0;
}
