"""Paged attention at the edges of what a call may hold: starts that do not
ascend, many sequences, long lists of pages, values that are not finite
(tests/decode_reference.py holds the derivation of the tolerances)."""
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


@pytest.mark.parametrize("seqs", [128, 129, 300, 1100])
@pytest.mark.parametrize("kind,hq,hk,dim", [("bf16", 2, 1, 64), ("e4m3", 4, 2, 48)])
@pytest.mark.parametrize("chunks", [0, 1, 2])
def test_many_sequences(seqs, kind, hq, hk, dim, chunks):
    # past 128 sequences lengths are read again for each unit; single tokens alone, with a few chunks, with long ones
    g = torch.Generator().manual_seed(seqs + chunks)
    q_lens = (torch.rand(seqs, generator=g) < 0.9).int().tolist()
    kv_lens = torch.randint(0, 70, (seqs,), generator=g).tolist()
    for b in range(5, seqs, 60):
        q_lens[b] = [1, 40, 130][chunks]
        kv_lens[b] = q_lens[b] + 25
    q_lens[-1], kv_lens[-1] = q_lens[5], 500
    p = Problem(seqs, q_lens, kv_lens, hq, hk, dim, 16, kind)
    print("case", seqs, kind, hq, hk, dim, chunks, flush=True)
    p.check(p.run())
    if chunks:
        p.check(p.run(window=37), window=37)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,dim,kv,page", [(1, 64, 60000, 1), (1, 48, 60001, 1), (4, 64, 60013, 1), (40, 64, 30000, 1),
                                               (300, 48, 25000, 1), (1, 64, 240000, 2)])
def test_runs_of_more_pages_than_the_list_holds(kind, q_len, dim, kv, page):
    # a work-group's run reaches over more than 1024 pages
    p = Problem(kv + q_len, [q_len], [kv], 8 if q_len == 300 else 1, 1, dim, page, kind)
    print("case", kind, q_len, dim, kv, page, flush=True)
    if q_len < 300:
        p.check(p.run(scale=0.5), scale=0.5)
        return
    # (the definition of some rows: each as a call of its own prefix would give it)
    out, lse = p.run()
    rows = [0, 1, 170, 298, 299]
    clean = [torch.nan_to_num(t.float().double(), nan=0.0, posinf=0.0, neginf=0.0) for t in (p.k, p.v)]
    for i in rows:
        want = ref.attention(p.q[i:i + 1].double(), *clean, p.table.tolist(), [0, 1], [kv - q_len + i + 1], dim ** -0.5, 0,
                             p.ks, p.vs)
        tol, lse_tol = ref.attention_tolerance(*want, dim)
        assert ((out[i].double() - want[0][0]).abs() <= tol[0]).all()
        assert ((lse[i].double() - want[1][0]).abs() <= lse_tol[0]).all()


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("q_len,kv,key,window", [(4, 90, 88, 0), (5, 700, 697, 0), (4, 300, 255, 43), (2, 90, 50, 39),
                                                 (60, 190, 150, 0), (60, 190, 140, 33)])
@pytest.mark.parametrize("name", ["k", "v"])
def test_nan_of_an_8_bit_cache_reaches_its_rows_alone(dim, q_len, kv, key, window, name):
    p = Problem(31, [q_len], [kv], 4, 2, dim, 16, "e4m3")
    clean = p.run(window=window)
    _poisoned(p, 0, key, [0, 1], {name: float("nan")})
    print("case", dim, q_len, kv, key, window, name, flush=True)
    got = p.run(window=window)
    own = kv - q_len + torch.arange(q_len)
    sees = (own >= key) & (own < key + window if window else own >= 0)
    assert sees.any() and not sees.all()
    assert torch.isnan(got[0][sees].float()).all()
    assert torch.equal(got[0][~sees].view(torch.int16), clean[0][~sees].view(torch.int16))
    assert torch.equal(got[1][~sees], clean[1][~sees])
