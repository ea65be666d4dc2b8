"""Paged attention at the edges of what a call may hold: starts that do not
ascend, many sequences, long lists of pages, values that are not finite
(tests/decode_reference.py holds the derivation of the tolerances)."""
import pytest

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
