"""Paged attention at the edges of what a call may hold: starts that do not
ascend, many sequences, long lists of pages, values that are not finite
(tests/decode_reference.py holds the derivation of the tolerances)."""
import pytest

import tests.decode_reference as ref
from tests.test_parity_gpu_attention import Problem
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


@pytest.mark.parametrize("q_len", [3, 50])
@pytest.mark.parametrize("second", [-(1 << 31), -(1 << 31) + 2, -1, 0, 1, 1 << 30])
def test_starts_that_do_not_ascend_write_no_other_rows(q_len, second):
    # sequence 0 begins at row q_len, where sequence 1's start lies anywhere; rows past `tokens` keep what they hold
    p = Problem(4, [q_len, q_len], [90, 70], 4, 2, 64, 16, "bf16")
    tokens, room = 2 * q_len, 4 * q_len
    out = torch.full((room, p.hq, p.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((room, p.hq), 7.0, device="cuda")
    q = torch.zeros(room, p.hq, p.dim, dtype=torch.bfloat16, device="cuda")
    q[:tokens] = p.q_dev
    starts = torch.tensor([q_len, second, tokens], dtype=torch.int32, device="cuda")
    n = Q.paged_attention_workspace_size(p.cache, tokens, p.hq, 2, 2 * q_len, 90)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    print("case", q_len, second, flush=True)
    Q.paged_attention(p.cache, q[:tokens], out[:tokens], starts, p.dev[1], p.dev[2], ws, 2 * q_len, 90, lse=lse[:tokens])
    torch.cuda.synchronize()
    assert (out[tokens:] == 7).all() and (lse[tokens:] == 7).all()
    if second <= q_len:                                  # sequence 0 has no rows
        assert (out[:max(second, 0)] == 7).all()


def test_a_workspace_of_the_largest_call_serves_smaller_ones():
    # bounds of the largest call: 300 tokens of up to 40 sequences with up to 900 keys
    problems = [Problem(3, [300], [900], 8, 1, 128, 16, "bf16"), Problem(3, [1] * 40, [300] * 40, 8, 1, 128, 16, "bf16"),
                Problem(3, [1], [900], 8, 1, 128, 16, "bf16"), Problem(3, [60, 1, 5], [200, 900, 77], 8, 1, 128, 16, "bf16")]
    n = Q.paged_attention_workspace_size(problems[0].cache, 300, 8, 40, 300, 900)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for p in problems:
        p.check(p.run(workspace=ws))


def _same_specials(got, want):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got == float("inf"), want == float("inf"))
    assert torch.equal(got == -float("inf"), want == -float("inf"))


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("q_len,kv,key", [(1, 90, 70), (4, 90, 88), (4, 700, 698), (40, 200, 190), (40, 200, 100),
                                          (130, 300, 171), (600, 700, 650)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("far", [0, 1])
def test_an_infinite_value_weighs_as_its_probability(dim, q_len, kv, key, value, far):
    # a value of infinity gives infinity to the rows that see it, and NaN (zero times infinity) where its
    # probability is zero, whether all rows of a tile see the key or only later ones
    p = Problem(9, [q_len], [kv], 4, 2, dim, 16, "bf16")
    p.q_dev.fill_(1.0)
    p.q = p.q_dev.cpu()
    page, row = int(p.table[0, key // 16]), key % 16
    scale = dim ** -0.5
    for cache_v, cache_k in ((p.cache.v, p.cache.k), (p.v, p.k)):
        cache_v[page, :, row] = value
        if far:
            cache_k[page, :, row] = -1000.0                # a score of -1000 dim^0.5
    print("case", dim, q_len, kv, key, value, far, flush=True)
    got = p.run()
    owned = [torch.where(t.float().isnan() | (t.float().abs() > 1e30), torch.zeros(()), t.float()).double()
             for t in (p.k, p.v)]
    owned[1][page, :, row] = value
    want = ref.attention(p.q.double(), owned[0], owned[1], p.table.tolist(), p.q_start, p.kv_lens, scale)
    _same_specials(got[0], want[0])
    sees = kv - q_len + torch.arange(q_len) >= key
    assert sees.any() and (torch.isnan(got[0][sees].float()) if far else got[0][sees].float() == value).all()
