"""Sampling at the edges of its parameters against the 64-bit definition:
tokens must be equal."""
import numpy as np
import pytest

import tests.decode_reference as ref
from tests.test_parity_gpu_long_rows import _draw
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


def _want(logits, u, **opts):
    # beside infinity nothing else is drawn: such a row is one of zeros at its infinities and nothing elsewhere
    logits = logits.copy()
    for row in logits:
        if (row == np.inf).any() and not np.isnan(row).any():
            row[:] = np.where(row == np.inf, np.float32(0), np.float32(-np.inf))
    return ref.sample(logits, u, **opts)


# rows of one work-group, and of several
@pytest.mark.parametrize("n", [300, 5000, 40000])
@pytest.mark.parametrize("opts", [{}, {"top_k": 7}, {"top_k": 20000}, {"top_p": 0.5}, {"top_p": 0.9, "top_k": 100}, {"min_p": 0.5}])
def test_infinite_temperature(n, opts):
    # every finite logit weighs the same, one of -infinity nothing, and beside +infinity only that counts
    rng = np.random.default_rng(n)
    rows = (3 * rng.standard_normal((7, n))).astype(np.float32)
    rows[0, rng.random(n) < 0.97] = -np.inf
    rows[1, :-3] = -np.inf
    rows[2, 1:] = -np.inf
    rows[3, [n // 3, n // 2]] = np.inf
    rows[4, [5, n - 1]] = np.inf
    rows[4, 7:n // 2] = -np.inf
    rows[5] = np.round(rows[5])                       # thousands of equal logits
    rows[6] = np.where(rng.random(n) < 0.6, np.float32(1.0), np.float32(-np.inf))
    for t in (np.inf, 3e38):
        settings = {k: [v] * 7 for k, v in dict(opts, temperature=t).items()}
        for u in (0.0, 0.31, 0.77, 0.99999994):
            us = np.full(7, u, np.float32)
            print("case", n, opts, t, u, flush=True)
            assert np.array_equal(_draw(rows, us, **settings), _want(rows, us, **settings))


def test_a_workspace_of_the_largest_batch_serves_smaller_ones():
    n = 9000
    rng = np.random.default_rng(1)
    ws = torch.zeros(Q.sample_workspace_size(200, n), dtype=torch.uint8, device="cuda")
    idx = torch.empty(200, dtype=torch.int32, device="cuda")
    logits = (3 * rng.standard_normal((200, n))).astype(np.float32)
    x, u = torch.from_numpy(logits).cuda(), rng.random(200).astype(np.float32)
    for m, k in ((200, n), (128, n), (64, n), (1, n), (129, 8193), (3, 8192)):
        Q.sample_f32(x[:m, :k], torch.from_numpy(u[:m]).cuda(), idx[:m], ws)
        torch.cuda.synchronize()
        rows = sorted({0, m // 2, m - 1})
        assert np.array_equal(idx.cpu().numpy()[rows], ref.sample(logits[rows, :k], u[rows])), (m, k)
