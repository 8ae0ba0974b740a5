"""The host's choice between units of one and of two query tiles (sliding-window
prefill), compiled from the library's header by itself.  The choice changes no
result, only the time."""
import ctypes
import os
import subprocess

import pytest

from paged_kv_cache_174_gb300 import build as pkg_build

SOURCE = """
#include "pa_internal.h"
extern "C" int pairs(int tokens, int seqs, int min_q, int max_q, int tile, int n_kv, int sms,
                     double cost) {
  return pa::pairs_finish_sooner(tokens, seqs, min_q, max_q, tile, n_kv, sms, cost);
}
"""


@pytest.fixture(scope="module")
def pairs(tmp_path_factory):
    d = tmp_path_factory.mktemp("pair_rule")
    (d / "rule.cpp").write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(pkg_build.nvcc()))),
                        "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", pkg_build.CSRC, "-I",
                    pkg_build.INCLUDE, "-I", cuda, str(d / "rule.cpp"), "-o", str(d / "rule.so")],
                   check=True)
    f = ctypes.CDLL(str(d / "rule.so")).pairs
    f.argtypes = [ctypes.c_int] * 7 + [ctypes.c_double]

    def call(q_lens, group=4, n_kv=8, fp8=False, min_q=0):
        return bool(f(sum(q_lens), len(q_lens), min_q, max(q_lens), 128 // group, n_kv, 152,
                      1.45 if fp8 else 1.7))
    return call


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_requests_within_one_tile_have_no_pairs(pairs, fp8):
    for rows in (1, 2, 4, 31, 32):
        assert not pairs([rows] * 256, fp8=fp8)
        assert not pairs([rows] * 256, fp8=fp8, min_q=rows)
    assert not pairs([128] * 300, group=1, fp8=fp8)
    assert not pairs([16] * 3000, group=8, n_kv=1, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_rows_are_not_counted(pairs, fp8):
    """A chunk's choice is the same alone and beside any number of decodes."""
    for rows in (64, 512, 600):
        for decodes in (0, 1, 128, 300, 1000):
            assert not pairs([1] * decodes + [rows], fp8=fp8), (rows, decodes)
    for rows in (700, 1024, 2048, 8192):
        for decodes in (0, 1, 128, 300, 1000):
            assert pairs([1] * decodes + [rows], fp8=fp8), (rows, decodes)


def test_the_measured_shapes(pairs):
    assert not pairs([1300]) and pairs([1300], fp8=True)
    assert pairs([512] * 2) and pairs([512] * 4) and pairs([64] * 32) and pairs([128] * 16)
    assert not pairs([512] + [4] * 100, min_q=4)
    assert not pairs([512] + [4] * 100, min_q=4, fp8=True)
    for q_lens in ([48] * 64, [100] * 40, [64] * 32, [1024]):  # all alike: said or not
        assert pairs(q_lens) and pairs(q_lens, min_q=q_lens[0])
    assert not pairs([300] * 8) and pairs([300] * 8, fp8=True)
    assert pairs([1024], group=8, n_kv=8) and not pairs([1024], group=8, n_kv=2)
    assert not pairs([2048], group=1) and pairs([3000], group=1)


def test_degenerate_calls(pairs):
    assert not pairs([1]) and not pairs([0]) and not pairs([0] * 2000 + [1000])
    assert pairs([2 ** 31 - 1], n_kv=8)
