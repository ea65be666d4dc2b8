"""Arithmetic that keeps the decode kernels inside their buffers, on the host:
the functions that the kernels call, compiled for the CPU."""
import ctypes
import itertools
import random
import subprocess

import pytest

from tests.test_decode_ops_host import BAD, _attention, _cache, _rope_append
from weight_only_block_amd import build
from weight_only_block_amd import qgemv as Q

SOURCE = r"""
#include "decode_ops.h"
#include "rows.h"
extern "C" void cut_seq(int start, int next, int kv, int tokens, int max_q, int cap, int* out)
{
    const qg::Seq s = qg::cut_seq(start, next, kv, tokens, max_q, cap);
    out[0] = s.q0, out[1] = s.n, out[2] = s.kv;
}
extern "C" int rows_disjoint(int n, const int64_t* count, const int64_t* stride, int64_t width)
{
    qg::Dim two[2] = {{count[0], stride[0]}, {count[1], stride[1]}};
    if (n == 2) return qg::rows_disjoint(two, width);
    qg::Dim three[3] = {two[0], two[1], {count[2], stride[2]}};
    return qg::rows_disjoint(three, width);
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


def _disjoint(host, counts, strides, width):
    array = ctypes.c_int64 * len(counts)
    host.rows_disjoint.argtypes = [ctypes.c_int, array, array, ctypes.c_int64]
    return bool(host.rows_disjoint(len(counts), array(*counts), array(*strides), width))


def test_rows_share_no_element(host):
    # small layouts, nested or not, against every pair of rows
    rng = random.Random(0)
    seen = {True: 0, False: 0}
    for _ in range(20000):
        n, width = rng.choice([2, 3]), rng.choice([1, 2, 4])
        counts, strides = [rng.randint(1, 5) for _ in range(n)], [rng.randint(0, 40) for _ in range(n)]
        starts = sorted(sum(i * s for i, s in zip(at, strides)) for at in itertools.product(*[range(c) for c in counts]))
        want = all(b - a >= width for a, b in zip(starts, starts[1:]))
        assert _disjoint(host, counts, strides, width) == want, (counts, strides, width)
        seen[want] += 1
    assert min(seen.values()) > 2000
    top = 1 << 31
    assert not _disjoint(host, [top - 1, 65535, 1 << 20], [top, 16, 1 << 20], 16)  # 2048 slots on is the next page
    assert _disjoint(host, [top - 1, 1 << 15, 1 << 12], [top, 16, 1 << 19], 16)    # nested, past 2^61 elements
    assert not _disjoint(host, [top - 1, 65535, 1 << 20], [16, 16, 16], 16)
    assert not _disjoint(host, [top - 1, 65535], [16, 32], 16)
    assert _disjoint(host, [9, 2], [128, 1088], 64)                               # crosses, in the gaps


def test_overlapping_rows_are_refused():
    row = dict(head_stride=64, slot_stride=64)
    for over in (row, dict(slot_stride=64, head_stride=128), dict(slot_stride=256, head_stride=64, page_stride=64),
                 dict(page_stride=1024), dict(page_stride=4032), dict(slot_stride=192, head_stride=64)):
        c = _cache(**over)
        assert _rope_append(cache=c) == BAD and _attention(cache=c) == BAD, over
        assert Q.lib().qg_paged_attention_workspace_size(ctypes.addressof(c), 3, 8, 2, 2, 100) == 0
    # slots outside heads, pages innermost, padded rows; a dimension of one entry has no stride
    for over in (dict(slot_stride=256, head_stride=64), dict(page_stride=64, head_stride=9 * 64, slot_stride=36 * 64),
                 dict(slot_stride=72, head_stride=1152, page_stride=4608), dict(kv_heads=1, head_stride=64),
                 dict(pages=1, page_stride=0)):
        c = _cache(**over)
        assert Q.lib().qg_paged_attention_workspace_size(ctypes.addressof(c), 3, 8, 2, 2, 100) > 0, over
    for token, head in ((64, 64), (448, 64), (64, 128), (128, 64)):
        assert _rope_append(_13=token, _14=head) == BAD, (token, head)
        assert _attention(_4=token, _5=head) == BAD, (token, head)
