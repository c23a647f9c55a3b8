"""csrc/device_once.h, compiled on its own with a fake of the failing call:
what failed is asked again, what succeeded is not, each device for itself."""
import os
import subprocess

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_once.h"

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

enum Error { kOk = 0, kPending = 4, kTooFew = 9 };

int main() {
    static pa::DeviceOnce<2, 3> once;
    int calls = 0;
    Error next = kPending;
    auto ask = [&] { ++calls; return next; };
    CHECK(once.run(0, 1, ask) == kPending && calls == 1);  // another call's pending error
    next = kOk;
    CHECK(once.run(0, 1, ask) == kOk && calls == 2);       // ... does not stay
    next = kTooFew;
    CHECK(once.run(0, 1, ask) == kOk && calls == 2);       // a success does
    CHECK(once.run(1, 1, ask) == kTooFew && calls == 3);   // on its device alone
    CHECK(once.run(0, 2, ask) == kTooFew && calls == 4);   // and for its kernel
    next = kOk;
    for (int k = 0; k < 2; ++k)                            // outside the table: every time
        CHECK(once.run(2, 0, ask) == kOk && once.run(-1, 0, ask) == kOk && once.run(0, 3, ask) == kOk);
    CHECK(calls == 10);
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t) threads.emplace_back([&] { once.run(1, 0, ask); });
    for (auto &t : threads) t.join();
    CHECK(calls == 11);
    return 0;
}
"""


def test_only_success_is_remembered(tmp_path):
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_attention_decode_split_gb300",
                        "csrc")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-pthread", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
