// once_check.cc -- OncePerDevice on the host, with setters that count and fail.
#include <cstdio>
#include <thread>
#include <vector>

#include "gdn_device.h"

int main() {
  static gdn::OncePerDevice once;
  int calls[100] = {};
  auto run = [&](int dev, int rc) {
    return once.run(dev, [&] { ++calls[dev]; return rc; });
  };
  if (run(0, 0) != 0 || run(0, 0) != 0 || calls[0] != 1) return 1;      // once on a device
  if (run(1, 0) != 0 || calls[1] != 1) return 2;                         // and on the next one
  if (run(2, -8) != -8 || run(2, -8) != -8 || calls[2] != 2) return 3;  // a failure is not kept
  if (run(2, 0) != 0 || run(2, -8) != 0 || calls[2] != 3) return 4;
  if (run(70, 0) != 0 || run(70, 0) != 0 || calls[70] != 2) return 5;   // past the known ones: always
  if (run(0, -8) != 0) return 6;
  std::atomic<int> sets{0}, bad{0};
  std::vector<std::thread> ts;
  for (int i = 0; i < 8; ++i)
    ts.emplace_back([&] {
      for (int k = 0; k < 1000; ++k)
        if (once.run(5, [&] { ++sets; return 0; }) != 0) ++bad;
    });
  for (auto& t : ts) t.join();
  if (bad != 0 || sets < 1 || sets > 8) return 7;
  std::printf("ok\n");
  return 0;
}
