"""Order of the device status codes (csrc/device_status.h): a wait that gave up is never hidden by
an input error.  A CTA's word and a call's are the largest rank of what was recorded; here of codes
written by hand."""
import itertools
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# the code reported for the codes in argv
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "device_status.h"

int main(int argc, char** argv) {
  uint32_t top = 0;
  for (int i = 1; i < argc; ++i) {
    const uint32_t rank = nabla::status_rank(static_cast<uint32_t>(strtoul(argv[i], nullptr, 16)));
    top = rank > top ? rank : top;
  }
  printf("%x %d\n", nabla::status_of_rank(top), nabla::is_timeout_rank(top));
  return 0;
}
"""
TIMEOUTS, INPUT = ("101", "105", "10a"), ("301", "302")


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("status")
    (d / "main.cpp").write_text(PROGRAM)
    inc = os.path.join(ROOT, "adaptive_block_sparse_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", inc, str(d / "main.cpp"), "-o", str(d / "main")],
                   check=True, capture_output=True, text=True)

    def largest(*codes):
        out = subprocess.run([str(d / "main"), *codes], check=True, capture_output=True, text=True).stdout.split()
        return out[0], out[1] == "1"
    return largest


def test_a_timeout_is_reported_before_input_errors(run):
    assert run("0", "0") == ("0", False)
    for t in TIMEOUTS:
        assert run(t) == (t, True) and run("0", t) == (t, True)
    for e in INPUT:
        assert run(e) == (e, False) and run(e, "0", e) == (e, False)
    for t, e in itertools.product(TIMEOUTS, INPUT):
        for words in itertools.permutations(("0", t, e, e)):
            assert run(*words) == (t, True)


def test_the_kernels_codes_are_told_apart(run):
    """Every code of a wait is a timeout by its number; those of the inputs are not."""
    text = "".join(open(os.path.join(ROOT, "adaptive_block_sparse_b200", "csrc", f)).read()
                   for f in ("common.cuh", "history.cuh"))
    codes = dict(re.findall(r"(kDev\w+) = 0x([0-9A-Fa-f]+)", text))
    assert {"kDevTimeoutTmaFull", "kDevTimeoutDrain", "kDevBadPage", "kDevBadLength"} <= codes.keys()
    for name, code in codes.items():
        if name.startswith(("kDevTimeout", "kDevBad")):
            assert run(code) == (code.lower(), name.startswith("kDevTimeout"))
