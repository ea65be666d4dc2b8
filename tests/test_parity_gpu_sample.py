"""Sampling on the GPU against the 64-bit definition: tokens must be equal."""
import numpy as np
import pytest

import tests.decode_reference as ref
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


def _run(logits, u, ws=None, pad=0, **opts):
    logits = np.asarray(logits, np.float32)
    m, n = logits.shape
    x = torch.full((m, n + pad), 1e30, device="cuda")[:, :n]
    x.copy_(torch.from_numpy(logits))
    idx = torch.full((m,), -5, dtype=torch.int32, device="cuda")
    ws = torch.zeros(Q.sample_workspace_size(m, n), dtype=torch.uint8, device="cuda") if ws is None else ws
    dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
           for k, v in opts.items() if v is not None}
    Q.sample_f32(x, torch.tensor(u, dtype=torch.float32, device="cuda"), idx, ws, **dev)
    torch.cuda.synchronize()
    return idx.cpu().numpy()


def _options(rng, m, kind):
    pick = lambda vals: [float(rng.choice(vals)) for _ in range(m)]
    return {"temperature": pick([0.3, 0.7, 1.0, 2.0]) if kind != "none" else None,
            "top_k": [int(rng.choice([1, 2, 20, 1000])) for _ in range(m)] if "k" in kind else None,
            "top_p": pick([0.0, 0.1, 0.8, 0.95, 0.999]) if "p" in kind else None,
            "min_p": pick([0.01, 0.1, 1.0, 2.0]) if "m" in kind else None}


@pytest.mark.parametrize("m,n", [(1, 1), (3, 2), (5, 63), (4, 1000), (9, 4097), (2, 32001), (17, 8192), (3, 151936)])
@pytest.mark.parametrize("kind", ["none", "t", "k", "p", "kp", "m", "kpm"])
def test_sample_random_rows(m, n, kind):
    rng = np.random.default_rng([m, n, sum(map(ord, kind))])
    logits = 2.5 * rng.standard_normal((m, n))
    logits[:, rng.integers(0, n, 8)] += 6
    u = rng.random(m).astype(np.float32)
    opts = _options(rng, m, kind)
    print("case", m, n, kind, flush=True)
    assert np.array_equal(_run(logits, u, pad=int(rng.integers(0, 3)), **opts), ref.sample(logits, u, **opts))


@pytest.mark.parametrize("n", [257, 40000])
def test_sample_ties_and_clusters(n):
    # few distinct values, all equal, two far clusters, huge ranges, denormals
    rng = np.random.default_rng(n)
    rows = [rng.integers(-3, 4, n).astype(np.float64), np.full(n, 7.25), np.where(rng.random(n) < 0.5, 1e4, 1e4 - 1),
            rng.standard_normal(n) * 1e30, rng.standard_normal(n) * 1e-40, np.linspace(-1, 1, n) * 1e-3,
            np.where(np.arange(n) % 2 == 0, 0.0, -0.0), 100.0 + rng.integers(0, 2, n) * 2.0 ** -17]
    logits = np.stack(rows)
    m = len(rows)
    for top_k in (None, 1, 50, n - 1, n, n + 9):
        for top_p in (None, 0.0, 0.5, 0.9):
            u = rng.random(m).astype(np.float32)
            opts = {"top_k": None if top_k is None else [top_k] * m, "top_p": None if top_p is None else [top_p] * m,
                    "temperature": [float(rng.choice([0.05, 1.0, 5.0])) for _ in range(m)]}
            print("case", n, top_k, top_p, flush=True)
            assert np.array_equal(_run(logits, u, **opts), ref.sample(logits, u, **opts)), (top_k, top_p)


def test_sample_masked_nan_and_infinite_rows():
    rng = np.random.default_rng(11)
    n = 5000
    rows = rng.standard_normal((8, n)) * 3
    rows[0] = -np.inf
    rows[1] = -np.inf
    rows[1, 4321] = -7
    rows[2, [77, 99]] = np.nan
    rows[3, [5, 4000]] = np.inf
    rows[4, rng.random(n) < 0.97] = -np.inf
    rows[5] = np.finfo(np.float32).min
    rows[6] = np.finfo(np.float32).min
    rows[6, 100:110] = 0.5
    rows[7, 1:] = -np.inf
    for u in (0.0, 0.3, 0.99999994):
        for opts in ({}, {"top_k": [40] * 8}, {"top_p": [0.9] * 8}, {"top_k": [4] * 8, "min_p": [0.5] * 8},
                     {"temperature": [0.0, 1.0, 0.0, 1.0, 0.0, 1.0, 0.0, 1.0]}):
            us = np.full(8, u, np.float32)
            print("case", u, sorted(opts), flush=True)
            assert np.array_equal(_run(rows, us, **opts), ref.sample(rows, us, **opts))


def test_sample_extreme_uniforms_and_parameters():
    rng = np.random.default_rng(4)
    logits = rng.standard_normal((6, 3000)) * 4
    top = logits.argmax(1)
    u = np.array([0.0, 0.5, 0.25, 0.75, 0.1, 0.9], np.float32)
    # u = 0 takes the first kept token, however small its weight
    zero = np.zeros(6, np.float32)
    assert np.array_equal(_run(logits, zero), np.zeros(6, np.int32))
    # u of 1 or NaN, negative or NaN temperature: the greedy choice
    assert np.array_equal(_run(logits, np.ones(6, np.float32)), top)
    assert np.array_equal(_run(logits, np.full(6, np.nan, np.float32)), top)
    for t in (0.0, -1.0, float("nan")):
        assert np.array_equal(_run(logits, u, temperature=[t] * 6), top)
    # NaN cuts are none; negative top_k is none; a vanishing temperature is the greedy choice
    want = ref.sample(logits, u)
    assert np.array_equal(_run(logits, u, top_p=[float("nan")] * 6, min_p=[float("nan")] * 6, top_k=[-3] * 6), want)
    assert np.array_equal(_run(logits, u, temperature=[1e-30] * 6), top)


def test_sample_distribution():
    # frequencies over even uniforms are the weights, to one part in m
    n, m = 9, 4096
    x = np.linspace(-1.0, 1.5, n)
    u = ((np.arange(m) + 0.5) / m).astype(np.float32)
    got = np.bincount(_run(np.tile(x, (m, 1)), u), minlength=n)
    p = np.exp(np.float64(np.float32(x)))
    p /= p.sum()
    assert np.abs(got / m - p).max() <= 1.5 / m


def test_sample_repeats_shares_a_workspace_and_replays_in_a_graph():
    rng = np.random.default_rng(8)
    ws = torch.zeros(Q.sample_workspace_size(20, 60000), dtype=torch.uint8, device="cuda")
    for m, n in ((20, 60000), (3, 1000), (1, 60000), (20, 5)):
        logits = rng.standard_normal((m, n)) * 3
        u = rng.random(m).astype(np.float32)
        opts = _options(rng, m, "kpm")
        assert np.array_equal(_run(logits, u, ws=ws, **opts), ref.sample(logits, u, **opts))
    m, n = 4, 20000
    x = torch.zeros(m, n, device="cuda")
    u = torch.zeros(m, device="cuda")
    top_p = torch.full((m,), 0.9, device="cuda")
    idx = torch.zeros(m, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        Q.sample_f32(x, u, idx, ws, top_p=top_p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        Q.sample_f32(x, u, idx, ws, top_p=top_p)
    for i in range(4):
        logits = rng.standard_normal((m, n)) * (2 + i)
        us = rng.random(m).astype(np.float32)
        x.copy_(torch.from_numpy(logits))
        u.copy_(torch.from_numpy(us))
        graph.replay()
        torch.cuda.synchronize()
        got = idx.cpu().numpy()
        assert np.array_equal(got, ref.sample(logits, us, top_p=[0.9] * m))
        assert np.array_equal(_run(logits, us, ws=ws, top_p=[0.9] * m), got)
