"""What a launch keeps of each device (compiled for the host; no GPU)."""
import ctypes as C
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_opt_decode_b200", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("per_device")
    (d / "p.cpp").write_text(
        '#include "per_device.h"\n'
        "static flexq::PerDevice kept;\nstatic int asked;\n"
        'extern "C" int get(int dev, int answer, int error, int* value) {\n'
        "  return kept.get(dev, value, [&](int* v) { ++asked; *v = answer; return error; });\n}\n"
        'extern "C" int count() { return asked; }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC, str(d / "p.cpp"), "-o",
                    str(d / "p.so")], check=True)
    return C.CDLL(str(d / "p.so"))


def test_each_device_has_its_own_value_and_failures_are_not_kept(lib):
    def get(dev, answer, error=0):
        v = C.c_int(-1)
        return lib.get(dev, answer, error, C.byref(v)), v.value
    assert get(0, 148) == (0, 148) and get(1, 132) == (0, 132)
    assert get(0, 7) == (0, 148) and get(1, 7) == (0, 132) and lib.count() == 2
    assert get(2, 0, 3)[0] == 3  # the error of the query
    assert get(2, 96) == (0, 96) and get(2, 7) == (0, 96) and lib.count() == 4
    assert get(64, 5) == (0, 5) and get(64, 6) == (0, 6) and get(-1, 4) == (0, 4) and lib.count() == 7


def test_no_launch_keeps_a_number_for_all_devices():
    """Function-local statics of the serving kernels are arrays by device or PerDevice."""
    for name in ("attn_paged.cu", "attn_paged_chunk.cu", "gemv_q4.cu", "paged_append.cu", "warp_mma.cuh"):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for line in re.findall(r"^ +static (?!constexpr|_assert)[^\n]*", src, re.M):
            assert re.match(r" +static (PerDevice \w+(\[[^\]]*\])?|std::atomic<int> allowed\[64\]);", line), (name, line)
