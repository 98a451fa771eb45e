"""What the library keeps for each device, on the CPU: a program that counts calls, and the sources."""
import pathlib
import re
import subprocess

CSRC = pathlib.Path(__file__).parents[1] / "gated_deltanet_linear_build_gb300" / "csrc"

PROGRAM = r"""
#include <cstdio>
#include "per_device.h"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
enum Status { kOk, kFailed };
int calls = 0;
Status result = kOk;
Status set(int device) {                 // a library's function: its state is a static of its own
  static gdn::DeviceOnce once;
  return once(device, [] { ++calls; return result; });
}
int found = 0;
int number(int device) {
  static gdn::DeviceNumber n;
  return n(device, [] { ++calls; return found; });
}
int main() {
  result = kFailed;
  CHECK(set(0) == kFailed && set(0) == kFailed && calls == 2);        // a failure is not kept
  result = kOk;
  CHECK(set(0) == kOk && set(0) == kOk && calls == 3);                // a success is, on its device
  result = kFailed;
  CHECK(set(0) == kOk && set(1) == kFailed && calls == 4);
  result = kOk;
  CHECK(set(1) == kOk && set(63) == kOk && calls == 6 && set(63) == kOk && set(0) == kOk && calls == 6);
  CHECK(set(64) == kOk && set(64) == kOk && set(-1) == kOk && set(-1) == kOk && calls == 10);
  calls = 0;
  CHECK(number(3) == 0 && number(3) == 0 && calls == 2);
  found = 152;
  CHECK(number(3) == 152 && number(3) == 152 && calls == 3);
  found = 8;
  CHECK(number(0) == 8 && number(3) == 152 && number(0) == 8 && calls == 4);
  CHECK(number(-1) == 8 && number(-1) == 8 && number(1000) == 8 && calls == 7);
  return 0;
}
"""


def test_each_device_is_asked_once(tmp_path):
    src = tmp_path / "t.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "t"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", str(CSRC), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_function_keeps_what_belongs_to_a_device():
    for path in sorted(CSRC.glob("*.cu*")):
        text = path.read_text()
        for m in re.finditer(r"static const [^;]*?(?:;|\}\(\);)", text, re.S):
            assert not re.search(r"cudaFuncSetAttribute|cudaDeviceGetAttribute|spread<|clusters_of", m.group(0)), \
                (path.name, m.group(0))
        for call in re.finditer(r"cudaFuncSetAttribute\(|cudaDeviceGetAttribute\(", text):
            before = text[max(0, call.start() - 700):call.start()]
            assert re.search(r"current_device\(\)|cudaError_t spread\(\)", before), (path.name, text[call.start():][:80])
