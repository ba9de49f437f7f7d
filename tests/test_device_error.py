"""The device error words as status and message, compiled for the host (no GPU needed)."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, CAPACITY, TIMEOUT = 0, -6, -7
EXTENT = 1 << 16

SRC = r"""
#include "device_error.h"
static std::string msg;
extern "C" int status(const unsigned* bits) {
  const fg::DeviceErrorWord w[4] = {{"GEMM", bits[0]}, {"ragged cache", bits[1]},
                                    {"windowed decode attention", bits[2]},
                                    {"windowed prefill attention", bits[3]}};
  return fg::device_error_status(w, 4, &msg);
}
extern "C" const char* message() { return msg.c_str(); }
extern "C" unsigned extent() { return fg::kErrExtent; }
"""


@pytest.fixture(scope="module")
def dll(tmp_path_factory):
    d = tmp_path_factory.mktemp("device_error")
    src, lib = d / "e.cpp", d / "e.so"
    src.write_text(SRC)
    inc = os.path.join(ROOT, "bit_compressed_throughput_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o",
                    str(lib)], check=True)
    dll = C.CDLL(str(lib))
    dll.message.restype = C.c_char_p
    return dll


@pytest.mark.parametrize("bits,status,parts,absent", [
    ((0, 0, 0, 0), OK, [], []),
    ((2, 0, 0, 0), TIMEOUT, ["GEMM flag 2"], ["windowed", "fit"]),
    ((4, 0, 0, 0), TIMEOUT, ["GEMM flag 4"], ["fit"]),
    ((0, 0, 1, 0), TIMEOUT, ["windowed decode attention flag 1"], ["GEMM", "fit"]),
    ((0, EXTENT, 0, 0), CAPACITY, ["ragged cache", "does not fit"], ["timed out", "GEMM"]),
    ((0, 0, EXTENT, EXTENT), CAPACITY, ["windowed decode attention, windowed prefill attention"],
     ["timed out"]),
    ((1, EXTENT, 0, 3), TIMEOUT, ["GEMM flag 1", "windowed prefill attention flag 3",
                                  "does not fit", "ragged cache"], []),
    ((0, 0, EXTENT | 2, 0), TIMEOUT, ["windowed decode attention flag 2", "does not fit"], []),
])
def test_every_error_is_told(dll, bits, status, parts, absent):
    """Reading the words clears them, so a timeout does not hide an extent that did not fit, and
    each kernel family is named for its own."""
    assert dll.extent() == EXTENT
    assert dll.status((C.c_uint * 4)(*bits)) == status
    if status != OK:
        text = dll.message().decode()
        assert all(p in text for p in parts) and not any(a in text for a in absent), text
