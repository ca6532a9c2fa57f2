"""The shared-memory limit of a kernel, raised by launches on several host
threads at once (csrc/optin.h, compiled here with the host compiler)."""
import subprocess

from fft_long_convolution_flashconv_b200 import build

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

#include "optin.h"

using namespace std::chrono_literals;

int main() {
  {  // a small request is inside the setting call while a large one arrives
    fc::RaisedLimit limit;
    std::atomic<size_t> attribute{0};
    std::atomic<bool> inside{false}, large_done{false};
    std::thread small([&] {
      limit.raise(0, 34, [&](size_t n) {
        inside = true;
        for (int i = 0; i < 200 && !large_done; ++i) std::this_thread::sleep_for(1ms);
        attribute = n;
        return 0;
      });
    });
    while (!inside) std::this_thread::sleep_for(1ms);
    limit.raise(0, 94, [&](size_t n) { attribute = n; return 0; });
    large_done = true;
    small.join();
    if (attribute != 94) return std::printf("lowered to %zu\n", attribute.load()), 1;
    bool again = false;
    limit.raise(0, 94, [&](size_t) { again = true; return 0; });
    limit.raise(0, 34, [&](size_t) { again = true; return 0; });
    if (again) return std::printf("set again\n"), 1;
  }
  for (int device : {0, 63, 64, 1000}) {  // never downwards, whatever the order
    fc::RaisedLimit limit;
    std::atomic<size_t> attribute{0};
    std::atomic<bool> lowered{false};
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
      threads.emplace_back([&, t] {
        for (size_t i = 1; i <= 200; ++i) {
          const size_t want = (i * 37 + t * 101) % 211 + 1;
          limit.raise(device, want, [&](size_t n) {
            if (n <= attribute) lowered = true;
            attribute = n;
            return 0;
          });
          if (attribute < want) lowered = true;
        }
      });
    for (auto& t : threads) t.join();
    if (lowered) return std::printf("device %d: lowered\n", device), 1;
  }
  {  // a refused size leaves the limit, and devices do not share one
    fc::RaisedLimit limit;
    int calls = 0;
    if (limit.raise(1, 50, [&](size_t) { ++calls; return 7; }) != 7) return std::printf("status lost\n"), 1;
    if (limit.raise(1, 50, [&](size_t) { ++calls; return 0; }) != 0) return 1;
    limit.raise(2, 50, [&](size_t) { ++calls; return 0; });
    if (calls != 3) return std::printf("%d calls\n", calls), 1;
  }
  return std::puts("ok"), 0;
}
"""


def test_limit_is_never_lowered(tmp_path):
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True, timeout=60)
    assert (run.returncode, run.stdout) == (0, "ok\n")
