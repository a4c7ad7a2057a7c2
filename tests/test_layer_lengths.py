"""The layer operators' arithmetic on row lengths, up to the 2^31 - 1 tokens a
call may have, compiled for the host with overflow checks.  No GPU is used."""
from __future__ import annotations

import os
import subprocess

from gated_deltanet_linear_gdr_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_linear_gdr_gb300", "csrc", "layer")

PROGRAM = r"""
#include "layer_internal.h"
#include <stdio.h>
int main() {
    const int lengths[] = {-1, 0, 1, 63, 64, 65, 1 << 30, 2147483583, 2147483584, 2147483585, 2147483646, 2147483647};
    const int sizes[] = {1, 4, 64, 256, 64 * 524288, 1 << 30, 2147483647};
    for (int n : lengths)
        for (int s : sizes) printf("%d %d %d\n", n, s, gdr::pieces(n, s));
    return 0;
}
"""


def test_pieces_of_rows(tmp_path):
    src, exe = tmp_path / "pieces.cc", tmp_path / "pieces"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(libbuild._nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                    "-fsanitize-undefined-trap-on-error", "-I", CSRC, "-isystem", cuda, str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(lines) == 84
    for line in lines:
        n, size, got = map(int, line.split())
        assert got == (0 if n <= 0 else -(-n // size)), line


def test_no_row_length_is_rounded_up_by_adding():
    """(len + size - 1) / size wraps for the longest rows; pieces() does not."""
    import re
    for name in sorted(os.listdir(CSRC)):
        if name.startswith("k_la_"):
            with open(os.path.join(CSRC, name)) as f:
                for i, line in enumerate(f, 1):
                    assert not re.search(r"(len|s_len\[\w+\]|row_len\[\w+\]).{0,6}\+ \(?(kC|c\.seg|kT|kTok) - 1", line), f"{name}:{i}"
