"""Attention over the paged cache on the GPU against the 64-bit definition
(tests/decode_reference.py holds the derivation of the tolerances)."""
import math

import pytest

import tests.decode_reference as ref
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


class Problem:
    """Inputs on the host and the device.  Cache slots that no sequence owns
    hold NaN and infinities, table entries past a sequence's pages hold -1."""

    def __init__(self, seed, q_lens, kv_lens, hq, hk, dim, page, kind, nhd=False, qkv_rows=False, magnitude=1.0):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.dim, self.hq, self.hk, self.page = q_lens, kv_lens, dim, hq, hk, page
        need = [-(-kv // page) for kv in kv_lens]
        pages = sum(need) + 2
        cols = max(max(need), 1)
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(kv_lens), cols), -1, dtype=torch.int32)
        shape = (pages, page, hk, dim) if nhd else (pages, hk, page, dim)
        k, v = magnitude * torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        if nhd:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        self.ks = self.vs = None
        if kind == "bf16":
            k, v = k.bfloat16(), v.bfloat16()
        else:
            self.ks = 0.01 + 0.02 * torch.rand(hk, generator=g)
            self.vs = 0.01 + 0.02 * torch.rand(hk, generator=g)
            k, v = (60 * k).clamp(-448, 448).to(torch.float8_e4m3fn), (60 * v).clamp(-448, 448).to(torch.float8_e4m3fn)
        owned = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for b, kv in enumerate(kv_lens):
            for c in range(need[b]):
                table[b, c] = order[at]
                owned[order[at], :min(page, kv - c * page)] = True
                at += 1
        # foreign slots hold what must not be seen
        stale = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e38]).repeat(-(-dim // 4))[:dim]
        if kind != "bf16":
            stale = torch.where(torch.isfinite(stale), torch.tensor(448.0), torch.tensor(float("nan")))
        raw = torch.int16 if kind == "bf16" else torch.uint8
        bits = stale.to(k.dtype).view(raw)
        for t in (k, v):
            for p, s in (~owned).nonzero().tolist():
                t.view(raw)[p, :, s] = bits
        self.k, self.v, self.table = k, v, table
        self.q_start = [0]
        for n in q_lens:
            self.q_start.append(self.q_start[-1] + n)
        tokens = self.q_start[-1]
        wide = torch.randn(tokens, hq + 2 * hk if qkv_rows else hq, dim, generator=g).bfloat16()
        self.q = wide[:, :hq]
        self.q_dev = wide.cuda()[:, :hq]
        self.cache = Q.KVCache(k.cuda(), v.cuda(), None if self.ks is None else self.ks.cuda(),
                               None if self.vs is None else self.vs.cuda())
        self.dev = [torch.tensor(self.q_start, dtype=torch.int32, device="cuda"),
                    torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), table.cuda()]
        self.max_q, self.max_kv = max(q_lens + [1]), max(kv_lens + [1])

    def run(self, scale=None, window=0, workspace=None, max_q=None, max_kv=None):
        tokens = self.q_start[-1]
        max_q, max_kv = max_q or self.max_q, max_kv or self.max_kv
        out = torch.full((tokens, self.hq, self.dim), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((tokens, self.hq), 7.0, device="cuda")
        if workspace is None:
            n = Q.paged_attention_workspace_size(self.cache, tokens, self.hq, len(self.q_lens), max_q, max_kv)
            workspace = torch.zeros(n, dtype=torch.uint8, device="cuda")
        Q.paged_attention(self.cache, self.q_dev, out, *self.dev, workspace, max_q, max_kv, scale=scale,
                          window=window, lse=lse)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def want(self, scale=None, window=0):
        clean = [torch.nan_to_num(t.float().double(), nan=0.0, posinf=0.0, neginf=0.0) for t in (self.k, self.v)]
        return ref.attention(self.q.double(), clean[0], clean[1], self.table.tolist(), self.q_start, self.kv_lens,
                             self.dim ** -0.5 if scale is None else scale, window, self.ks, self.vs)

    def check(self, got, scale=None, window=0):
        out, lse, spread, slack = self.want(scale, window)
        tol, lse_tol = ref.attention_tolerance(out, lse, spread, slack, self.dim)
        got_out, got_lse = got[0].double(), got[1].double()
        empty = lse == -math.inf
        assert (got_lse[empty] == -math.inf).all() and (got_out[empty] == 0).all()
        err = (got_out - out).abs()
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
        assert ((got_lse - lse).abs()[~empty] <= lse_tol[~empty]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim,page", [
    (16, 8, 128, 16), (8, 8, 64, 16), (14, 2, 64, 32), (40, 8, 128, 64), (24, 4, 80, 16), (6, 2, 96, 1),
    (8, 1, 256, 32), (3, 1, 16, 8), (2, 2, 48, 128), (5, 1, 112, 16), (48, 1, 128, 16), (4, 2, 160, 4), (2, 1, 240, 2)])
@pytest.mark.parametrize("kv_lens", [[1], [5, 0, 64, 65], [127, 700, 31, 1, 300]])
def test_single_tokens(kind, hq, hk, dim, page, kv_lens):
    print("case", kind, hq, hk, dim, page, kv_lens, flush=True)
    p = Problem(1 + dim + page + len(kv_lens), [1] * len(kv_lens), kv_lens, hq, hk, dim, page, kind)
    p.check(p.run())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim,page", [(8, 2, 128, 16), (7, 1, 64, 32), (4, 4, 80, 16), (2, 1, 256, 64), (3, 1, 96, 8)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([5, 3, 1], [400, 3, 90]), ([0, 2, 0, 9], [10, 2, 0, 333]), ([7], [4]), ([70, 1, 33], [70, 500, 200]),
    ([130], [135]), ([1, 200, 0, 3, 64], [257, 300, 64, 1, 64])])
def test_chunks(kind, hq, hk, dim, page, q_lens, kv_lens):
    print("case", kind, hq, hk, dim, page, q_lens, kv_lens, flush=True)
    p = Problem(7 + dim + sum(q_lens), q_lens, kv_lens, hq, hk, dim, page, kind, nhd=dim == 128, qkv_rows=dim == 64)
    p.check(p.run())


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 10000])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 65]), ([66, 1, 5], [190, 129, 40])])
def test_windows(window, q_lens, kv_lens):
    for kind, hq, hk, dim in (("bf16", 6, 2, 64), ("e4m3", 4, 1, 128)):
        print("case", window, q_lens, kv_lens, kind, flush=True)
        p = Problem(window, q_lens, kv_lens, hq, hk, dim, 16, kind)
        p.check(p.run(window=window), window=window)


def test_freed_pages_before_a_window():
    # pages wholly before every window may be gone from the table
    p = Problem(3, [1, 4], [400, 320], 4, 2, 64, 16, "bf16")
    p.dev[2][0, :(400 - 50) // 16] = -1
    p.dev[2][1, :(320 - 3 - 50) // 16] = -1
    p.check(p.run(window=50), window=50)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 40])
def test_long_sequences_split_over_the_chip(kind, q_len):
    for hq, hk, dim, kv in ((4, 1, 128, 9001), (2, 2, 64, 16000)):
        p = Problem(kv + q_len, [q_len, 1], [kv, 77], hq, hk, dim, 32, kind)
        print("case", kind, q_len, kv, flush=True)
        p.check(p.run())


def test_scores_far_apart():
    # scores of some thousands: one key takes all the weight, nothing overflows
    p = Problem(5, [3, 1], [333, 700], 4, 2, 64, 16, "bf16", magnitude=300.0)
    p.check(p.run(scale=2.0), scale=2.0)
    p.check(p.run(scale=-2.0), scale=-2.0)
    p.check(p.run(scale=0.0), scale=0.0)


def _poisoned(p, table_pos, key, heads, where):
    """Writes a value into one key's K or V row; returns nothing."""
    page, row = int(p.table[table_pos, key // p.page]), key % p.page
    for name, value in where.items():
        t = getattr(p.cache, name)
        for h in heads:
            t[page, h, row] = torch.full((p.dim,), value, device="cuda").to(t.dtype)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_len,kv,key", [(40, 200, 190), (4, 90, 88), (130, 300, 171), (70, 70, 69)])
def test_unseen_keys_do_not_reach_a_row(dim, q_len, kv, key):
    # a key that only later tokens see holds NaN or infinity: rows before it are as if it held zeros
    for name, value in (("v", float("nan")), ("v", float("inf")), ("k", float("nan")), ("k", float("inf"))):
        p = Problem(9, [q_len], [kv], 4, 2, dim, 16, "bf16")
        clean = p.run()
        _poisoned(p, 0, key, [0, 1], {name: value})
        print("case", dim, q_len, kv, key, name, value, flush=True)
        got = p.run()
        before = key - (kv - q_len)                 # rows that do not see the key
        assert torch.equal(got[0][:before], clean[0][:before]) and torch.equal(got[1][:before], clean[1][:before])
        if name == "v":
            assert not torch.isfinite(got[0][before:].float()).any()
        elif value != value:
            assert torch.isnan(got[0][before:].float()).all()


@pytest.mark.parametrize("window", [9, 33])
def test_keys_before_a_window_do_not_reach_a_row(window):
    p = Problem(9, [20], [150], 4, 2, 64, 16, "bf16")
    clean = p.run(window=window)
    key = 150 - 20 - window + 8                     # in the window of the first rows alone
    _poisoned(p, 0, key, [0, 1], {"v": float("nan")})
    got = p.run(window=window)
    sees = [key > 130 + i - window for i in range(20)]
    for i, s in enumerate(sees):
        if s:
            assert torch.isnan(got[0][i].float()).all()
        else:
            assert torch.equal(got[0][i], clean[0][i])


def test_a_query_of_nan_stays_in_its_row():
    for q_len in (3, 50):
        p = Problem(2, [q_len], [120], 4, 2, 64, 16, "bf16")
        clean = p.run()
        p.q_dev[1, 2] = float("nan")
        got = p.run()
        assert torch.isnan(got[0][1, 2].float()).all()
        got[0][1, 2] = clean[0][1, 2]
        assert torch.equal(got[0], clean[0])


def test_lengths_are_cut_to_the_bounds():
    # kv_len past the table or max_kv, and q_start past `tokens`, read nothing beyond
    p = Problem(4, [2, 3], [64, 48], 4, 2, 64, 16, "bf16")
    full = p.run()
    p.dev[1][0] = 1 << 30
    p.dev[0][2] = 1 << 30
    got = p.run()
    assert torch.equal(got[0], full[0])
    p.dev[1][0] = -5
    got = p.run()
    assert (got[0][:2] == 0).all() and torch.equal(got[0][2:], full[0][2:])


def test_pages_outside_the_cache_count_as_nan():
    for bad in (-1, 1 << 30, -(1 << 31)):
        for q_len in (1, 40):
            p = Problem(4, [q_len, 1], [200, 90], 4, 2, 64, 16, "bf16")
            full = p.run()
            p.dev[2][0, 3] = bad
            print("case", bad, q_len, flush=True)
            got = p.run()
            assert torch.isnan(got[0][:q_len].float()).all()
            assert torch.equal(got[0][q_len:], full[0][q_len:])


def test_same_bits_again_whatever_ran_before_in_the_workspace():
    small = Problem(1, [1] * 5, [300, 20, 900, 1, 77], 8, 2, 128, 16, "bf16")
    large = Problem(2, [150, 1], [700, 1200], 8, 2, 128, 16, "e4m3")
    size = max(Q.paged_attention_workspace_size(p.cache, p.q_start[-1], p.hq, len(p.q_lens), p.max_q, p.max_kv)
               for p in (small, large))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = [p.run(workspace=ws) for p in (small, large)]
    for _ in range(3):
        for p, want in zip((large, small), reversed(first)):
            got = p.run(workspace=ws)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # wider bounds than needed still hold
    small.check(small.run(max_q=9, max_kv=5000))


def test_calls_of_many_shapes_share_a_workspace():
    # what one shape leaves behind its counts must not be another's counts
    problems = [Problem(10 + i, [q] * n, [kv] * n, hq, 2, dim, 16, kind) for i, (q, n, kv, hq, dim, kind) in enumerate([
        (1, 2, 3000, 4, 128, "bf16"), (40, 3, 700, 4, 64, "e4m3"), (1, 70, 90, 2, 64, "bf16"), (3, 1, 4000, 8, 256, "e4m3"),
        (200, 1, 900, 2, 128, "bf16"), (1, 1, 9000, 4, 80, "bf16")])]
    want = [p.run() for p in problems]
    size = max(Q.paged_attention_workspace_size(p.cache, p.q_start[-1], p.hq, len(p.q_lens), p.max_q, p.max_kv)
               for p in problems)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    order = torch.Generator().manual_seed(0)
    for _ in range(5):
        for i in torch.randperm(len(problems), generator=order).tolist():
            got = problems[i].run(workspace=ws)
            assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1]), i


def test_replays_in_a_graph():
    p = Problem(6, [1, 1, 1], [500, 33, 900], 8, 2, 128, 16, "bf16")
    tokens = 3
    out = torch.zeros(tokens, p.hq, p.dim, dtype=torch.bfloat16, device="cuda")
    n = Q.paged_attention_workspace_size(p.cache, tokens, p.hq, 3, 1, 900)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    call = lambda: Q.paged_attention(p.cache, p.q_dev, out, *p.dev, ws, 1, 900)
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for i, lens in enumerate(([500, 33, 900], [400, 1, 899], [1, 30, 70])):
        p.dev[1].copy_(torch.tensor(lens, dtype=torch.int32))
        p.kv_lens = lens
        p.q_dev.mul_(-1.0)
        p.q = p.q_dev.cpu()
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu()
        eager = p.run(workspace=ws, max_kv=900)
        assert torch.equal(got, eager[0])
        p.check(eager)


def test_offsets_past_32_bits():
    # the last pages of a cache of more than 2^31 elements
    hk, page, dim = 8, 128, 128
    pages = (1 << 31) // (hk * page * dim) + 9
    k = torch.zeros(pages, hk, page, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    last = list(range(pages - 3, pages))
    for t in (k, v):
        t[last] = torch.randn(3, hk, page, dim, generator=g, device="cuda").bfloat16()
    cache = Q.KVCache(k, v)
    q = torch.randn(1, 16, dim, generator=g, device="cuda").bfloat16()
    out = torch.zeros_like(q)
    table = torch.tensor([last], dtype=torch.int32, device="cuda")
    ws = torch.zeros(Q.paged_attention_workspace_size(cache, 1, 16, 1, 1, 300), dtype=torch.uint8, device="cuda")
    Q.paged_attention(cache, q, out, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                      torch.tensor([300], dtype=torch.int32, device="cuda"), table, ws, 1, 300)
    torch.cuda.synchronize()
    small_k, small_v = k[last].cpu().double(), v[last].cpu().double()
    want, lse, spread, slack = ref.attention(q.cpu().double(), small_k, small_v, [[0, 1, 2]], [0, 1], [300], dim ** -0.5)
    tol, _ = ref.attention_tolerance(want, lse, spread, slack, dim)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    # and the append reaches them
    slot = torch.tensor([(pages - 1) * page + page - 1], device="cuda")
    src = torch.ones(1, 16 + 2 * hk, dim, device="cuda")
    Q.rope_append(cache, Q.Rope(dim), src[:, :16], src[:, 16:16 + hk], src[:, 16 + hk:],
                  torch.zeros(1, dtype=torch.int32, device="cuda"), slot, out)
    torch.cuda.synchronize()
    assert (k[-1, :, -1] == 1).all() and (v[-1, :, -1] == 1).all()
