"""The arithmetic of a document's segments (csrc/decay_parts.h), compiled for the CPU."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT
from sparse_spatial_hashing_amd import prediction

MOST = 2**31 - 4096  # tokens of a call
WIDEST = 65536       # tokens of a segment


@pytest.fixture(scope="module")
def part_end(tmp_path_factory):
    work = tmp_path_factory.mktemp("parts")
    source, made = work / "parts.cpp", work / "parts.so"
    source.write_text('#include "decay_parts.h"\n'
                      'extern "C" int part(int from, int n, int segment) { return part_end(from, n, segment); }\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sparse_spatial_hashing_amd", "csrc"), str(source), "-o", str(made)], check=True)
    return ctypes.CDLL(str(made)).part


def test_segments_end_with_their_document(part_end):
    for n in (0, 1, 127, 128, 129, WIDEST, 2**31 - WIDEST - 1, 2**31 - WIDEST, 2**31 - WIDEST + 1, MOST - 1, MOST):
        for segment in (128, 160, WIDEST):
            whole = n // segment
            for p in {0, 1, whole // 2, max(0, whole - 1), whole}:
                if p * segment <= n:
                    assert part_end(p * segment, n, segment) == min(n, (p + 1) * segment), (n, segment, p)


def test_the_longest_document_reaches_the_widest_segments():
    """What the sizes above stand for: one head, as many tokens as a call takes."""
    a = prediction._Decay(dtype=1, heads=1, kv_heads=1, width=8, t=MOST, docs=1, decay=4096, scale=1.0,
                          q_stride=(8, 8), k_stride=(8, 8), v_stride=(8, 8), g_stride=(8, 8))
    assert prediction._lib.tok_decay_carry_rows(ctypes.byref(a)) == MOST // WIDEST
