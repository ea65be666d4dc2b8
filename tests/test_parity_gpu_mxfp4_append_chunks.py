"""The 4-bit append at chunk sizes: past 1024 rounds of heads (tokens x rounds)
a work-group takes all rounds of a token, queries, then keys, then values.  The
checks and their tolerances are those of test_parity_gpu_mxfp4_cache.py."""
import pytest

import tests.mxfp4_reference as mx
import tests.test_parity_gpu_mxfp4_cache as base
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


CASES = [
    # tokens, q heads, kv heads, dim, rot, page, source, interleaved, scaling, qkv in one row, order, odd exponents
    # eight dimensions a thread: halves, whole heads and parts of them, keys and values within a round and across two
    (400, 32, 8, 128, 128, 16, "f32", 0, None, 1, "phsd", 0),
    (400, 40, 8, 128, 64, 16, "bf16", 0, "yarn", 1, "pshd", 0),
    (300, 16, 8, 256, 192, 32, "bf16", 0, None, 0, "phsd", 1),
    (300, 21, 11, 256, 256, 16, "f32", 0, "linear", 1, "phsd", 0),
    (600, 60, 9, 64, 64, 16, "bf16", 0, None, 1, "phsd", 3),
    # and neighbours
    (300, 33, 17, 96, 96, 16, "f32", 1, None, 1, "phsd", 0),
    (300, 33, 17, 224, 40, 16, "bf16", 1, "yarn", 1, "hpsd", 0),
    # four dimensions a thread: more heads than a round holds, rot_dim off its vectors
    (300, 24, 12, 96, 48, 16, "f32", 0, None, 1, "phsd", 0),
    (200, 20, 20, 128, 96, 16, "bf16", 0, "linear", 1, "pshd", 0),
    (150, 70, 70, 64, 30, 8, "f32", 0, None, 1, "shpd", 0),
    (200, 17, 9, 160, 6, 8, "bf16", 1, None, 1, "phsd", 5),
    (200, 9, 9, 256, 254, 16, "f32", 0, "yarn", 0, "phsd", 0),
]


def rounds_of(case):
    """Rounds of heads and whether threads hold eight dimensions, for rows on 16 bytes."""
    _, hq, hk, dim, rot, _, _, inter = case[:8]
    eights = rot % 8 == 0 if inter else rot % 64 == 0 and dim % 64 == 0
    lanes = 256 // (dim // (8 if eights else 4))
    each = lambda heads: -(-heads // lanes)
    return each(hq + 2 * hk) if eights else each(hq) + 2 * each(hk)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("far", [0, 1])
def test_several_rounds_a_work_group(case, far):
    assert rounds_of(case) > 1 and case[0] * rounds_of(case) > 1024
    base.test_rope_append(case, far)


@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (30, False), (30, True)])
@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
def test_rows_off_16_bytes(rot, inter, src):
    # the same rows a row further on a grid of odd steps: the same bytes in the cache
    tokens, hq, hk, dim, page = 300, 20, 10, 128, 16
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(tokens, hq + 2 * hk, dim, generator=g).to(src).cuda()
    odd = torch.zeros(tokens, hq + 2 * hk, dim + 1, dtype=src, device="cuda")[..., 1:]
    odd.copy_(x)
    pages = tokens // page + 2
    slots = torch.randperm(pages * page, generator=g)[:tokens].cuda()
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g).int().cuda()
    rope = Q.Rope(rot, base=500000.0, interleaved=inter)
    got = []
    for heads in (x, odd):
        parts = [torch.zeros(pages, hk, page, n, dtype=torch.uint8, device="cuda") for n in (dim // 2, dim // 2, dim // 32, dim // 32)]
        q_out = torch.zeros(tokens, hq, dim + 1, dtype=torch.bfloat16, device="cuda")[..., 1:]
        if heads is x:
            q_out = q_out.contiguous()
        Q.rope_append(Q.KVCache(*parts), rope, heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:], pos, slots, q_out)
        torch.cuda.synchronize()
        got.append((parts, q_out.cpu().double()))
    for a, b in zip(got[0][0], got[1][0]):
        assert torch.equal(a, b)
    # (queries: each off by half a step of the output and some 2^-19 of its terms)
    y, z = got[0][1], got[1][1]
    assert ((y - z).abs() <= 2.0 ** -7 * y.abs() + 2.0 ** -18 * x[:, :hq].cpu().double().abs().amax(-1, keepdim=True)).all()


def test_keys_and_positions_past_the_first_launch():
    # a call of more than 2^23 tokens goes in several launches, each with its tokens' positions and slots
    tokens, dim = (1 << 23) + 5, 32
    row = torch.randn(1, 3, dim, generator=torch.Generator().manual_seed(4)).cuda()
    src = row.expand(tokens, 3, dim)
    parts = [torch.zeros(2, 1, 16, n, dtype=torch.uint8, device="cuda") for n in (dim // 2, dim // 2, 1, 1)]
    live = {0: (3, 5), 1 << 23: (31, 700), tokens - 1: (20, 70001)}            # token: slot, position
    slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    pos = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    for t, (slot, at) in live.items():
        slots[t], pos[t] = slot, at
    q_out = torch.zeros(tokens, 1, dim, dtype=torch.bfloat16, device="cuda")
    cache, rope = Q.KVCache(*parts), Q.Rope(dim)
    Q.rope_append(cache, rope, src[:, :1], src[:, 1:2], src[:, 2:], pos, slots, q_out)
    # the same three tokens as a call of their own
    few = torch.tensor(list(live))
    small = [torch.zeros_like(t) for t in parts]
    q_few = torch.zeros(3, 1, dim, dtype=torch.bfloat16, device="cuda")
    three = row.expand(3, 3, dim)
    Q.rope_append(Q.KVCache(*small), rope, three[:, :1], three[:, 1:2], three[:, 2:], pos[few.cuda()], slots[few.cuda()], q_few)
    torch.cuda.synchronize()
    for a, b in zip(parts, small):
        assert torch.equal(a, b)
    freq, _ = base.ref.rope_frequencies(dim, 10000.0)
    k, _ = base.ref.rotate(row[:, 1:2].cpu().double().expand(3, 1, dim), torch.tensor([p for _, p in live.values()]), freq, 1.0, dim, False)
    # (no rotated key within 2^-28 of a border at this seed: the definition's bytes)
    codes, exps = mx.encode(k)
    for i, (slot, _) in enumerate(live.values()):
        for t, want in ((parts[0], codes), (parts[2], exps)):
            assert torch.equal(t[slot // 16, 0, slot % 16].cpu(), want[i, 0])
    assert torch.equal(q_out[few.cuda()], q_few)
