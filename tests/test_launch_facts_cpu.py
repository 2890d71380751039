"""The launchers' per-device facts under several host threads: a key is never
found with another key's value, and a thread sanitizer sees no race."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ternary_weight_bit_bitlinear_b200", "csrc")

PROGRAM = """
#include <thread>
#include <vector>
#include "launch_facts.h"
static blh::KeyedFact fact;
static blh::CountFact count;
static blh::FlagFact flag;
static int lookup(int key) { return key * 7 - 100; }   // negative, zero and positive
int main() {
  int v = 0;
  if (fact.get(1, &v)) return 2;                       // nothing is known at first
  std::atomic<int> bad{0};
  std::vector<std::thread> ts;
  for (int t = 0; t < 4; ++t)
    ts.emplace_back([t, &bad] {
      for (int i = 0; i < 200000; ++i) {
        const int key = 1 + (i * (t + 1)) % 300000;
        int value = 0;
        if (!fact.get(key, &value)) fact.set(key, value = lookup(key));
        if (value != lookup(key)) bad = 1;
        const int other = 1 + i % 2;                    // two widths in turn
        if (!fact.get(other, &value)) fact.set(other, value = lookup(other));
        if (value != lookup(other)) bad = 1;
        if (count.load() == 0) count = 5;
        if (!flag) flag = true;
      }
    });
  for (auto& t : ts) t.join();
  fact.set(0x7fffffff, 0);                             // a value of zero is known too
  if (!fact.get(0x7fffffff, &v) || v != 0) return 3;
  return bad || count != 5 || !flag;
}
"""


@pytest.mark.parametrize("flags", [["-O2"], ["-O1", "-fsanitize=thread"]])
def test_facts_under_threads(tmp_path, flags):
    (tmp_path / "t.cc").write_text(PROGRAM)
    exe = str(tmp_path / "t")
    built = subprocess.run(["g++", "-std=c++17", "-pthread", "-I", CSRC, *flags,
                            str(tmp_path / "t.cc"), "-o", exe], capture_output=True, text=True)
    if built.returncode and "tsan" in built.stderr:
        pytest.skip("no thread sanitizer here")
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert ran.returncode == 0, ran.stderr[-2000:]


def test_every_fact_of_a_device_is_one_of_these():
    """DeviceInfo holds no plain word that a launcher writes: `sms` alone, which
    is written under a lock before anyone gets the structure."""
    src = open(os.path.join(CSRC, "internal.h")).read()
    body = src[src.index("struct DeviceInfo {"):]
    body = body[:body.index("\n};")]
    members = [l.split("//")[0].strip() for l in body.splitlines()[1:]]
    members = [m for m in members if m.endswith(";")]
    assert "int sms = 0;" in members
    members.remove("int sms = 0;")
    kinds = ("FlagFact ", "CountFact ", "KeyedFact ", "NormKernelInfo ")
    assert members and all(m.startswith(kinds) for m in members), members
    info = src[src.index("struct NormKernelInfo {"):]
    info = [l.strip() for l in info[:info.index("\n};")].splitlines()[1:]]
    assert info and all(l.startswith(kinds[:3]) for l in info), info
