"""Workspace sizes of the decode operators (no GPU): what serves a shape serves
every smaller one."""
import itertools

from weight_only_block_amd import qgemv as Q


def test_a_sampling_workspace_serves_smaller_calls():
    ms = [1, 2, 3, 16, 17, 64, 127, 128, 129, 200, 256, 257, 1000, 65535]
    ns = [1, 255, 4096, 4097, 8191, 8192, 8193, 9001, 12289, 32001, 151936, 262144, 262145, 600011, (1 << 31) - 1]
    size = {(m, n): Q.sample_workspace_size(m, n) for m, n in itertools.product(ms, ns)}
    for (m, n), (m2, n2) in itertools.product(size, size):
        if m2 <= m and n2 <= n:
            assert size[m2, n2] <= size[m, n], ((m2, n2), (m, n))
    assert Q.sample_workspace_size(0, 100) <= Q.sample_workspace_size(1, 1)
