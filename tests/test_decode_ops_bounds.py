"""Arithmetic that keeps the decode kernels inside their buffers, on the host:
the functions that the kernels call, compiled for the CPU."""
import ctypes
import itertools
import os
import subprocess

import pytest

from weight_only_block_amd import build

SOURCE = r"""
#include "decode_ops.h"
extern "C" void cut_seq(int start, int next, int kv, int tokens, int max_q, int cap, int* out)
{
    const qg::Seq s = qg::cut_seq(start, next, kv, tokens, max_q, cap);
    out[0] = s.q0, out[1] = s.n, out[2] = s.kv;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    folder = tmp_path_factory.mktemp("bounds")
    src, lib = folder / "bounds.cpp", folder / "bounds.so"
    src.write_text(SOURCE)
    subprocess.check_call([build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O2", "-shared", "-fPIC",
                           "-I", build.CSRC, str(src), "-o", str(lib)])
    return ctypes.CDLL(str(lib))


def test_sequences_stay_inside_the_call(host):
    # starts that do not ascend, lie outside the rows, or are any 32 bits: rows [q0, q0 + n) never leave [0, tokens)
    low, high = -(1 << 31), (1 << 31) - 1
    starts = [low, low + 1, low + 5, low + 6, -7, -1, 0, 1, 5, 6, 7, 8, 1000, high - 1, high]
    out = (ctypes.c_int * 3)()
    for tokens, max_q in ((1, 1), (7, 3), (7, 7), (7, high), (high, high)):
        for start, following in itertools.product(starts, starts):
            host.cut_seq(start, following, 5, tokens, max_q, 9, out)
            q0 = min(max(start, 0), tokens)
            n = min(max(min(max(following, 0), tokens) - q0, 0), max_q)
            assert (out[0], out[1]) == (q0, n), (tokens, max_q, start, following)
    for kv, cap in itertools.product([low, -1, 0, 3, 9, high], [0, 9, 1 << 30]):
        host.cut_seq(0, 1, kv, 1, 1, cap, out)
        assert out[2] == min(max(kv, 0), cap)
