"""State kept for each device (csrc/per_device.h), on the host: a small program
with a failing step and several device numbers; and that no kernel attribute or
residency query of the library is kept in a plain static."""
import glob
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_gemm_tiled_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "per_device.h"
using namespace gb300;
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
enum Err { OK = 0, BAD = 7 };
int main() {
  static OncePerDevice once;
  int calls[MAX_DEVICES] = {}, fail = 1;
  auto run = [&](int dev) { return once.run(dev, OK, [&] { calls[dev]++; return fail ? BAD : OK; }); };
  CHECK(run(0) == BAD && run(0) == BAD && calls[0] == 2);   // a failure is not kept
  fail = 0;
  CHECK(run(0) == OK && run(0) == OK && calls[0] == 3);     // a success is
  CHECK(run(1) == OK && run(MAX_DEVICES - 1) == OK);        // and each device has its own
  CHECK(calls[1] == 1 && calls[MAX_DEVICES - 1] == 1 && calls[0] == 3);
  fail = 1;
  CHECK(run(1) == OK && run(2) == BAD);

  static CountPerDevice counts;
  int asked = 0;
  auto get = [&](int dev, int n) { return counts.get(dev, [&] { ++asked; return n; }); };
  CHECK(get(0, -1) == 0 && get(0, 76) == 76 && get(0, 5) == 76 && asked == 2);
  CHECK(get(1, 0) == 0 && get(1, 9) == 0 && asked == 3);    // none is an answer
  CHECK(get(2, 12) == 12 && get(0, 1) == 76 && asked == 4);

  static OncePerDevice shared;
  std::atomic<int> steps{0};
  std::vector<std::thread> t;
  for (int i = 0; i < 8; ++i)
    t.emplace_back([&] { for (int d = 0; d < MAX_DEVICES; ++d) shared.run(d, OK, [&] { ++steps; return OK; }); });
  for (auto& x : t) x.join();
  CHECK(steps >= MAX_DEVICES && steps <= 8 * MAX_DEVICES);
  puts("ok");
}
"""


def test_state_of_each_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I" + CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.stdout == "ok\n", r.stdout


def test_no_device_state_in_a_plain_static():
    """An initialiser of a static runs for the device of the first call alone."""
    bad = []
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\bstatic\b[^;{}()]*=\s*(?:\[[^\]]*\]\s*\{)?", text):
            end = text.find("\n  }", m.end()) if m.group(0).endswith("{") else text.find(";", m.end())
            if re.search(r"cudaFuncSetAttribute|cudaOccupancy|cudaDeviceGetAttribute|resident_clusters",
                         text[m.start(): end]):
                bad.append((os.path.basename(path), m.group(0)))
        for m in re.finditer(r"\bstatic\s+(?:int|std::atomic<int>)\s+(\w+)[^;(]*;", text):
            if m.group(1) in ("slots", "sms", "n"):
                bad.append((os.path.basename(path), m.group(0)))
    assert not bad, bad
