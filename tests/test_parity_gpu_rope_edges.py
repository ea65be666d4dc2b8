"""Rotary positions with cache append at the edges of what a call may hold."""
import pytest

import tests.decode_reference as ref
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


@pytest.mark.parametrize("rot", [16, 6])
def test_more_tokens_than_one_launch_takes(rot):
    # a grid has fewer than 2^32 threads: 2^24 tokens of 256 threads each are one too many (both kernels)
    tokens, dim = (1 << 24) + 5, 16
    g = torch.Generator(device="cuda").manual_seed(rot)
    row = torch.randn(1, 3, dim, generator=g, device="cuda").bfloat16()
    src = row.expand(tokens, 3, dim)
    k = torch.zeros(2, 1, 16, dim, dtype=torch.bfloat16, device="cuda")
    cache = Q.KVCache(k, torch.zeros_like(k))
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    slots[0], slots[-1] = 3, 20
    q_out = torch.full((tokens, 1, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    print("case", rot, flush=True)
    Q.rope_append(cache, Q.Rope(rot), src[:, :1], src[:, 1:2], src[:, 2:], pos, slots, q_out)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, tokens - 1])
    freq, amp = ref.rope_frequencies(rot, 10000.0)
    for got, head in ((q_out[at.cuda()].cpu(), 0), (cache.k[[0, 1], :, [3, 4]].cpu(), 1)):
        where = at if head == 0 else at[[0, -1]]
        x = row[:, head:head + 1].cpu().double().expand(len(where), 1, dim)
        want, mag = ref.rotate(x, where, freq, amp, rot, False)
        slack = 2.0 ** -20 * mag
        assert ((got.double() - want).abs() <= ref.BF16_HALF * (want.abs() + slack) + slack).all()
    assert torch.equal(cache.v[[0, 1], :, [3, 4]], row[:, 2:3].expand(2, 1, dim))
    assert not (q_out == 7).all(-1).any()
