// Checks csrc/per_device.h; exits 0 when all hold.
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

#define REQUIRE(c)                                         \
  do {                                                     \
    if (!(c)) {                                            \
      std::printf("line %d: %s\n", __LINE__, #c);          \
      return 1;                                            \
    }                                                      \
  } while (0)

int main() {
  static moe::PerDevice set;
  int made = 0, v = 0;
  auto value = [&](int want, int error) {
    return [&made, want, error](int* out) {
      ++made;
      *out = want;
      return error;
    };
  };
  // one value a device, made once there
  REQUIRE(set.get(0, &v, value(10, 0)) == 0 && v == 10 && made == 1);
  REQUIRE(set.get(0, &v, value(11, 0)) == 0 && v == 10 && made == 1);
  REQUIRE(set.get(1, &v, value(20, 0)) == 0 && v == 20 && made == 2);
  REQUIRE(set.get(0, &v, value(11, 0)) == 0 && v == 10 && made == 2);
  REQUIRE(set.get(63, &v, value(30, 0)) == 0 && v == 30 && made == 3);
  // an error is not kept
  REQUIRE(set.get(2, &v, value(40, 7)) == 7 && made == 4);
  REQUIRE(set.get(2, &v, value(41, 0)) == 0 && v == 41 && made == 5);
  // outside the table: made every time
  REQUIRE(set.get(-1, &v, value(50, 0)) == 0 && v == 50 && made == 6);
  REQUIRE(set.get(64, &v, value(51, 0)) == 0 && v == 51 && made == 7);
  REQUIRE(set.get(64, &v, value(52, 0)) == 0 && v == 52 && made == 8);
  // host threads at once, four devices
  static moe::PerDevice shared;
  std::atomic<int> wrong{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 20000; ++i) {
        const int dev = (t + i) & 3;
        int got = 0;
        if (shared.get(dev, &got, [dev](int* out) { *out = 100 + dev; return 0; }) || got != 100 + dev)
          ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  REQUIRE(wrong == 0);
  return 0;
}
