// Drives the runtime's kept counts (kept_count.h) without CUDA: a query that fails
// is asked again, one that succeeded is not, devices and sizes are apart.
// Prints "ok" or the first check that does not hold.
#include <cstdio>

#include "kept_count.h"

#define CHECK(x)                               \
  if (!(x)) {                                  \
    std::printf("line %d: %s\n", __LINE__, #x); \
    return 1;                                  \
  }

enum Error { kNone = 0, kBusy = 2 };

int main() {
  static s2::KeptCounts<9> kept;
  int asked = 0, n = -7;
  auto fails = [&](int* m) {
    ++asked;
    *m = 5;
    return kBusy;
  };
  auto gives = [&](int value) {
    return [&asked, value](int* m) {
      ++asked;
      *m = value;
      return kNone;
    };
  };
  CHECK(kept.get(0, 8, &n, fails) == kBusy && asked == 1 && n == -7);
  CHECK(kept.get(0, 8, &n, gives(16)) == kNone && asked == 2 && n == 16);      // not taken for an answer of 0
  CHECK(kept.get(0, 8, &n, gives(3)) == kNone && asked == 2 && n == 16);
  CHECK(kept.get(0, 8, &n, fails) == kNone && asked == 2 && n == 16);
  CHECK(kept.get(1, 8, &n, gives(4)) == kNone && asked == 3 && n == 4);
  CHECK(kept.get(0, 7, &n, gives(0)) == kNone && asked == 4 && n == 0);        // none is an answer, too
  CHECK(kept.get(0, 7, &n, gives(1)) == kNone && asked == 4 && n == 0);
  for (int i = 0; i < 2; ++i) {                                                // beyond the table: asked every time
    CHECK(kept.get(16, 8, &n, gives(6)) == kNone && asked == 5 + i && n == 6);
  }
  std::printf("ok\n");
  return 0;
}
