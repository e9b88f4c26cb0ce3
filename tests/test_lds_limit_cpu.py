"""The dynamic-LDS limit of a kernel, on the host: a small program in which the two runtime calls
are its own, with two devices and a failure."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_only_offline_amd", "csrc")
ROCM = "/opt/rocm/include"

PROGRAM = r"""
#include "ql_lds_limit.hpp"
#include <cstdio>
static int device = 0, calls = 0;
static hipError_t answer = hipSuccess;
hipError_t hipGetDevice(int *d) { *d = device; return hipSuccess; }
hipError_t hipFuncSetAttribute(const void *, hipFuncAttribute, int bytes) { ++calls; return bytes == 4096 ? answer : hipErrorInvalidValue; }
int main() {
    ql::LdsLimit a, b;
    auto at = [&](ql::LdsLimit &k, int d, hipError_t says) {
        device = d;
        answer = says;
        const int before = calls;
        const hipError_t e = k.raise(&a, 4096);
        std::printf("%d:%d ", e == hipSuccess, calls - before);
    };
    at(a, 0, hipErrorOutOfMemory);   // a failure is reported
    at(a, 0, hipSuccess);            // and tried again
    at(a, 0, hipErrorOutOfMemory);   // raised: no further call
    at(a, 1, hipSuccess);            // another device needs its own
    at(a, 1, hipErrorOutOfMemory);
    at(a, 0, hipErrorOutOfMemory);
    at(b, 0, hipSuccess);            // another kernel too
    at(a, 64, hipSuccess);           // past the mask: every time
    at(a, 64, hipSuccess);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM), reason="needs g++ and the HIP headers")
def test_limit_is_raised_on_each_device_and_after_a_failure(tmp_path):
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-w", "-I", CSRC, "-I", ROCM, str(src), "-o", str(exe)],
                   check=True, timeout=100)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=10, check=True).stdout.split()
    assert out == ["0:1", "1:1", "1:0", "1:1", "1:0", "1:0", "1:1", "1:1", "1:1"]
