"""Attention of sequences with thousands of rows (tokens x query heads of a kv
head), where a work-group takes 256 rows at once, and sampling from rows of
more than 2^18 logits, against the 64-bit definitions (tests/decode_reference.py
holds the derivation of the tolerances; tokens must be equal)."""
import numpy as np
import pytest

import tests.decode_reference as ref
from tests.test_parity_gpu_attention import Problem, _poisoned
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim,page", [(8, 1, 128, 16), (9, 1, 64, 32), (8, 1, 80, 1), (16, 2, 96, 8), (8, 1, 48, 128),
                                            (8, 1, 112, 4), (8, 1, 256, 64), (8, 1, 160, 16)])
@pytest.mark.parametrize("q_lens,kv_lens", [([300], [300]), ([271], [700]), ([400, 0, 451], [401, 9, 900])])
def test_many_rows(kind, hq, hk, dim, page, q_lens, kv_lens):
    print("case", kind, hq, hk, dim, page, q_lens, kv_lens, flush=True)
    p = Problem(3 + dim + sum(q_lens), q_lens, kv_lens, hq, hk, dim, page, kind, nhd=dim == 128, qkv_rows=dim == 64)
    p.check(p.run())


@pytest.mark.parametrize("window", [1, 33, 64, 250])
@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3", 64)])
def test_many_rows_with_a_window(kind, dim, window):
    p = Problem(window, [300, 260], [300, 700], 8, 1, dim, 16, kind)
    print("case", kind, dim, window, flush=True)
    p.check(p.run(window=window), window=window)


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("key", [299, 431, 500])
def test_many_rows_do_not_see_later_keys(kind, dim, key):
    # a key that only later tokens see holds a value that is not finite: rows
    # before it keep their bits, rows that see a value of NaN give NaN
    q_len, kv = 260, 501
    for name in ("k", "v"):
        p = Problem(21, [q_len], [kv], 8, 1, dim, 16, kind)
        clean = p.run()
        _poisoned(p, 0, key, [0], {name: float("nan")})
        print("case", kind, dim, key, name, flush=True)
        out, lse = p.run()
        first = key - (kv - q_len)                   # the first token that sees it
        assert torch.equal(out[:first].view(torch.int16), clean[0][:first].view(torch.int16))
        assert torch.equal(lse[:first], clean[1][:first])
        assert torch.isnan(out[first:].float()).all()


def test_same_bits_whatever_stands_beside_a_long_sequence_in_the_workspace():
    p = Problem(5, [333], [900], 8, 1, 128, 16, "bf16")
    n = Q.paged_attention_workspace_size(p.cache, 333, 8, 1, 333, 900)
    workspace = torch.zeros(n, dtype=torch.uint8, device="cuda")
    one = p.run(workspace=workspace)
    for _ in range(3):
        two = p.run(workspace=workspace)
        assert torch.equal(one[0].view(torch.int16), two[0].view(torch.int16)) and torch.equal(one[1], two[1])


# ------------------------------------------------------------------- sampling

def _draw(logits, u, **opts):
    m, n = logits.shape
    idx = torch.full((m,), -5, dtype=torch.int32, device="cuda")
    ws = torch.full((Q.sample_workspace_size(m, n),), 0xa5, dtype=torch.uint8, device="cuda")
    dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in opts.items()}
    Q.sample_f32(torch.from_numpy(logits).cuda(), torch.from_numpy(u).cuda(), idx, ws, **dev)
    torch.cuda.synchronize()
    return idx.cpu().numpy()


def _settings(kind, m):
    opts = {"t": {"temperature": 0.9}, "k": {"top_k": 1000}, "p": {"top_p": 0.95, "temperature": 1.3},
            "kp": {"top_k": 300, "top_p": 0.9}, "m": {"min_p": 0.02}, "kpm": {"top_k": 50, "top_p": 0.99, "min_p": 0.05}}[kind]
    return {k: [v] * m for k, v in opts.items()}


@pytest.mark.parametrize("m,n", [(1, 262144), (2, 262145), (3, 300001), (2, 600011), (1, 1048583)])
@pytest.mark.parametrize("kind", ["t", "k", "p", "kp", "m", "kpm"])
def test_long_rows(m, n, kind):
    rng = np.random.default_rng([m, n, ord(kind[0])])
    logits = (2.5 * rng.standard_normal((m, n))).astype(np.float32)
    logits[:, rng.integers(0, n, 8)] += 6
    opts = _settings(kind, m)
    for u in (rng.random(m).astype(np.float32), np.full(m, 0.99999994, np.float32), np.zeros(m, np.float32)):
        print("case", m, n, kind, u[0], flush=True)
        assert np.array_equal(_draw(logits, u, **opts), ref.sample(logits, u, **opts))


def test_a_row_masked_but_for_its_ends():
    n = 300001
    logits = np.full((3, n), -np.inf, np.float32)
    logits[0, [0, n - 1]] = 1.0
    logits[1, n - 1] = -2.0
    logits[2, 511:513] = 3.0                          # both sides of a group's end
    for u in (0.0, 0.49, 0.51, 0.99999994):
        us = np.full(3, u, np.float32)
        for kind in ("t", "k", "p", "kpm"):
            opts = _settings(kind, 3)
            print("case", u, kind, flush=True)
            assert np.array_equal(_draw(logits, us, **opts), ref.sample(logits, us, **opts))


@pytest.mark.parametrize("n", [9001, 270001])
@pytest.mark.parametrize("kind", ["t", "kp", "p"])
def test_many_long_rows(n, kind):
    # a work-group a row; some of the rows are checked
    m = 130
    rng = np.random.default_rng(n)
    logits = rng.standard_normal((m, n), dtype=np.float32) * 3
    u = rng.random(m).astype(np.float32)
    opts = _settings(kind, m)
    print("case", n, kind, flush=True)
    got = _draw(logits, u, **opts)
    rows = [0, 1, 64, 128, 129]
    assert np.array_equal(got[rows], ref.sample(logits[rows], u[rows], **{k: v[:5] for k, v in opts.items()}))


def test_nearly_equal_logits():
    # thousands of tokens in the cut's bin
    rng = np.random.default_rng(2)
    logits = (0.01 * rng.standard_normal((3, 100000))).astype(np.float32)
    u = rng.random(3).astype(np.float32)
    for kind in ("k", "p", "kp", "kpm"):
        opts = _settings(kind, 3)
        print("case", kind, flush=True)
        assert np.array_equal(_draw(logits, u, **opts), ref.sample(logits, u, **opts))
