"""How near attention of few rows over a 4-bit cache comes to the 64-bit
definition.

With up to 32 rows a sequence and kv head its probabilities enter the second product as two bf16 numbers, the second what
rounding the first left: each is off by at most half a step of that, 2^-8 of
2^-8.  The other terms are those of tests/decode_reference.py: scores held in
fp32 (delta, in numerator and denominator), exp2, rescales and fp32 sums
(2^-13), and the output's one rounding to bf16.
"""
import pytest

import tests.decode_reference as ref
from tests.test_parity_gpu_mxfp4_attention import Problem
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


@pytest.mark.parametrize("hq,hk,dim,page", [(16, 8, 128, 16), (14, 2, 64, 32), (24, 4, 96, 16), (8, 2, 256, 16), (2, 2, 32, 4),
                                            (5, 1, 160, 16), (3, 1, 192, 16), (3, 1, 224, 1)])
@pytest.mark.parametrize("q_lens,kv_lens,window", [([1], [1023], 0), ([1, 1, 1], [1, 77, 700], 0), ([6, 2], [300, 1500], 0),
                                                   ([32, 1, 0, 4], [60, 500, 9, 200], 45)])
def test_only_the_output_is_rounded(hq, hk, dim, page, q_lens, kv_lens, window):
    q_lens = [min(n, 32 // (hq // hk)) for n in q_lens]
    print("case", hq, hk, dim, page, q_lens, window, flush=True)
    p = Problem(dim + len(q_lens), q_lens, kv_lens, hq, hk, dim, page)
    got = p.run(window=window)
    out, lse, spread, slack = p.want(window=window)
    delta = (dim + 4) * 2.0 ** -24 * slack
    rel = 2.0 ** -16 + 2.0 * delta + 2.0 ** -13
    tol = rel[..., None] * spread * (1 + ref.BF16_HALF) + ref.BF16_HALF * out.abs() + 2.0 ** -126
    err = (got[0].double() - out).abs()
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    p.check(got, window=window)
