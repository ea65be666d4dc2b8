"""The decode loop of examples/decode_step.py, each of its steps against the
64-bit definitions on what the step was given."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
import tests.decode_reference as ref
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_steps_match_the_definitions(example, kv):
    lengths = [37, 5, 70]
    block = example.Block(len(lengths), max(lengths) + 3, kv)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, example.VOCAB, (n,), generator=g).int().cuda() for n in lengths]

    def watch(block, logits, u, tokens, settings):
        torch.cuda.synchronize()
        last, cache = block.last, block.cache
        scales = [None if s is None else s.cpu() for s in (cache.k_scale, cache.v_scale)]
        want, lse, spread, slack = ref.attention(
            last["q"].cpu().double(), cache.k.cpu().float().double(), cache.v.cpu().float().double(),
            block.table.cpu().tolist(), last["starts"].tolist(), last["len"].tolist(), example.DIM ** -0.5, 0, *scales)
        tol, _ = ref.attention_tolerance(want, lse, spread, slack, example.DIM)
        assert ((last["out"].cpu().double() - want).abs() <= tol).all()
        host = {k: v.cpu().numpy() for k, v in settings.items()}
        assert np.array_equal(tokens.cpu().numpy(), ref.sample(logits.cpu().numpy(), u.cpu().numpy(), **host))

    got = example.generate(block, prompts, 3, watch=watch)
    assert got.shape == (3, len(lengths)) and ((got >= 0) & (got < example.VOCAB)).all()
    assert block.len.tolist() == [n + 3 - 1 for n in lengths]


def test_a_prompt_in_chunks_is_the_prompt_at_once(example):
    # the same prompt in one call, in three, and token by token
    g = torch.Generator().manual_seed(3)
    prompt = torch.randint(0, example.VOCAB, (53,), generator=g).int().cuda()
    results = []
    for cuts in ([53], [20, 1, 32], [1] * 53):
        block = example.Block(1, 60)
        at = 0
        for n in cuts:
            logits = block.forward(prompt[at:at + n], [n])
            at += n
        results.append((logits.cpu().double(), block.cache.k.cpu(), block.cache.v.cpu()))
    spread = results[0][0].abs().max()
    for logits, k, v in results[1:]:
        # projections of one row and of several take different kernels, each within 2e-3 of sum |w x|
        assert (logits - results[0][0]).abs().max() <= 0.05 * spread
        close = (k.double() - results[0][1].double()).abs()
        assert (close <= 0.02 * results[0][1].double().abs().max()).all()


def test_projections_are_the_library_gemv(example):
    block = example.Block(1, 16)
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((3, example.HIDDEN)).astype(np.float32)).bfloat16()
    y = block.project(block.qkv, x.cuda()).cpu().numpy()
    want, size = oracle.q8g64(block.qkv["q"], block.qkv["s"], x.view(torch.int16).numpy().view(np.uint16))
    assert oracle.within_tolerance(y.astype(np.float64), want, size, 2e-3).all()
