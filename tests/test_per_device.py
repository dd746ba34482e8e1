"""What the library finds out once a device (csrc/per_device.cuh), compiled for the host."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = r"""
#include <cassert>
#include "../routed_expert_layer_fp32_gb300/csrc/per_device.cuh"
int main() {
  static std::atomic<int> kept[moe::kMaxDevices];
  int calls = 0, answer = 152;
  auto find = [&] { ++calls; return answer; };
  assert(moe::once_a_device(kept, 0, find) == 152 && calls == 1);
  assert(moe::once_a_device(kept, 0, find) == 152 && calls == 1);   // kept
  answer = 132;
  assert(moe::once_a_device(kept, 1, find) == 132 && calls == 2);   // another device's own
  assert(moe::once_a_device(kept, 0, find) == 152 && moe::once_a_device(kept, 1, find) == 132 && calls == 2);
  answer = 0;
  assert(moe::once_a_device(kept, 2, find) == 0 && calls == 3);     // a failure is not kept
  answer = 7;
  assert(moe::once_a_device(kept, 2, find) == 7 && calls == 4);
  assert(moe::once_a_device(kept, -1, find) == 7 && moe::once_a_device(kept, moe::kMaxDevices, find) == 7 && calls == 6);
}
"""


def test_a_value_for_each_device(tmp_path):
    exe = str(tmp_path / "per_device")
    subprocess.run(["g++", "-std=c++17", "-O1", "-x", "c++", "-", "-I", HERE, "-o", exe], input=SOURCE, text=True, check=True)
    subprocess.run([exe], check=True)
