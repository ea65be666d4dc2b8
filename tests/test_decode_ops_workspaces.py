"""Workspace sizes of the decode operators (no GPU): what serves a shape serves
every smaller one."""
import ctypes
import itertools

import pytest

from weight_only_block_amd import qgemv as Q


def test_a_sampling_workspace_serves_smaller_calls():
    ms = [1, 2, 3, 16, 17, 64, 127, 128, 129, 200, 256, 257, 1000, 65535]
    ns = [1, 255, 4096, 4097, 8191, 8192, 8193, 9001, 12289, 32001, 151936, 262144, 262145, 600011, (1 << 31) - 1]
    size = {(m, n): Q.sample_workspace_size(m, n) for m, n in itertools.product(ms, ns)}
    for (m, n), (m2, n2) in itertools.product(size, size):
        if m2 <= m and n2 <= n:
            assert size[m2, n2] <= size[m, n], ((m2, n2), (m, n))
    assert Q.sample_workspace_size(0, 100) <= Q.sample_workspace_size(1, 1)


@pytest.mark.parametrize("hq,hk", [(8, 1), (16, 8), (40, 8), (48, 1)])
@pytest.mark.parametrize("dim,kind", [(64, Q.KV_BF16), (128, Q.KV_BF16), (128, Q.KV_E4M3), (256, Q.KV_BF16)])
def test_an_attention_workspace_serves_smaller_calls(hq, hk, dim, kind):
    cache = Q._CacheStruct(k=1 << 20, v=1 << 21, k_scale=1 << 22, v_scale=1 << 23, pages=1 << 20, page_stride=hk * 16 * dim,
                           head_stride=16 * dim, slot_stride=dim, kv_heads=hk, page_size=16, head_dim=dim, dtype=kind)
    ref, fn = ctypes.addressof(cache), Q.lib().qg_paged_attention_workspace_size
    tokens, seqs, max_q, max_kv = [1, 31, 302, 329, 2048, 9000], [1, 2, 40, 300], [1, 5, 33, 302, 9000], [1, 100, 5000, 1 << 20]
    size = {s: fn(ref, s[0], hq, s[1], s[2], s[3]) for s in itertools.product(tokens, seqs, max_q, max_kv)}
    assert min(size.values()) > 0
    for a, b in itertools.product(size, size):
        if all(x <= y for x, y in zip(a, b)):
            assert size[a] <= size[b], (a, b)
