"""The decode loop of examples/decode_step.py over a 4-bit cache, each of its
steps against the 64-bit definitions on what the step was given."""
import pytest

import tests.decode_reference as ref
import tests.mxfp4_reference as mx
from tests.test_example_decode_gpu import example  # noqa: F401 (a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_steps_match_the_definitions(example):  # noqa: F811
    lengths = [37, 5, 70]
    block = example.Block(len(lengths), max(lengths) + 3, "mxfp4")
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, example.VOCAB, (n,), generator=g).int().cuda() for n in lengths]

    def watch(block, logits, u, tokens, settings):
        torch.cuda.synchronize()
        last, cache = block.last, block.cache
        values = [mx.decode(c.cpu(), e.cpu()) for c, e in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        want, lse, spread, slack = ref.attention(last["q"].cpu().double(), *values, block.table.cpu().tolist(),
                                                 last["starts"].tolist(), last["len"].tolist(), example.DIM ** -0.5)
        tol, _ = ref.attention_tolerance(want, lse, spread, slack, example.DIM)
        assert ((last["out"].cpu().double() - want).abs() <= tol).all()

    got = example.generate(block, prompts, 3, watch=watch)
    assert got.shape == (3, len(lengths)) and ((got >= 0) & (got < example.VOCAB)).all()
    assert block.len.tolist() == [n + 3 - 1 for n in lengths]
    # what the cache holds of each sequence, read back
    cache = block.cache
    for b, n in enumerate(block.len.tolist()):
        where = [(int(block.table[b, i // example.PAGE]), i % example.PAGE) for i in range(n)]
        at = [torch.tensor(x) for x in zip(*where)]
        for rows, c, e in zip(block.cached(b, torch.float32), (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
            assert torch.equal(rows.cpu().double(), mx.decode(c.cpu()[at[0], :, at[1]], e.cpu()[at[0], :, at[1]]))
