"""Attention over a 4-bit cache on the GPU against the 64-bit definition over the
values that its codes stand for (tests/decode_reference.py holds the derivation
of the tolerances; codes are exact in bf16, so none is added)."""
import math

import pytest

import tests.mxfp4_reference as mx
import tests.test_parity_gpu_attention as base
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


class Problem(base.Problem):
    """Slots that no sequence owns hold NaN blocks and random codes, table
    entries past a sequence's pages hold -1."""

    def __init__(self, seed, q_lens, kv_lens, hq, hk, dim, page, nhd=False, qkv_rows=False, magnitude=1.0, odd=0):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.dim, self.hq, self.hk, self.page = q_lens, kv_lens, dim, hq, hk, page
        need = [-(-kv // page) for kv in kv_lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(kv_lens), max(max(need), 1)), -1, dtype=torch.int32)
        shape = (pages, page, hk, dim) if nhd else (pages, hk, page, dim)
        # blocks of many magnitudes
        spread = torch.exp2(torch.randint(-3, 4, shape[:3] + (dim // 32,), generator=g).float()).repeat_interleave(32, -1)
        x = [magnitude * torch.randn(shape, generator=g) * spread, torch.randn(shape, generator=g) * spread]
        owned = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for b, kv in enumerate(kv_lens):
            for c in range(need[b]):
                table[b, c] = order[at]
                owned[order[at], :min(page, kv - c * page)] = True
                at += 1
        held = owned[:, :, None, None] if nhd else owned[:, None, :, None]
        parts, values = [], []
        for t in x:
            codes, exps = mx.encode(t.double())
            codes = torch.where(held, codes, torch.randint(0, 256, codes.shape, generator=g).to(torch.uint8))
            exps = torch.where(held, exps, torch.randint(253, 256, exps.shape, generator=g).to(torch.uint8))
            values.append(mx.decode(codes, exps))
            wide = torch.full(exps.shape[:-1] + (exps.shape[-1] + odd,), 255, dtype=torch.uint8)
            wide[..., odd:] = exps
            parts += [codes.cuda(), wide.cuda()[..., odd:]]
        if nhd:
            parts, values = [t.transpose(1, 2) for t in parts], [t.transpose(1, 2) for t in values]
        self.k, self.v = values
        self.ks = self.vs = None
        self.cache = Q.KVCache(parts[0], parts[2], parts[1], parts[3])
        self.table = table
        self.q_start = [0]
        for n in q_lens:
            self.q_start.append(self.q_start[-1] + n)
        wide = torch.randn(self.q_start[-1], hq + 2 * hk if qkv_rows else hq, dim, generator=g).bfloat16()
        self.q, self.q_dev = wide[:, :hq], wide.cuda()[:, :hq]
        self.dev = [torch.tensor(self.q_start, dtype=torch.int32, device="cuda"),
                    torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), table.cuda()]
        self.max_q, self.max_kv = max(q_lens + [1]), max(kv_lens + [1])

    def set_exponent(self, seq, key, block, name, value):
        """One exponent byte of a key's or value's block, in all heads."""
        t = getattr(self.cache, name + "_scale")
        t[int(self.table[seq, key // self.page]), :, key % self.page, block] = value


@pytest.mark.parametrize("hq,hk,dim,page", [
    (16, 8, 128, 16), (8, 8, 64, 16), (14, 2, 64, 32), (40, 8, 128, 64), (24, 4, 96, 16), (6, 2, 96, 1),
    (8, 1, 256, 32), (3, 1, 32, 8), (2, 2, 64, 128), (5, 1, 160, 16), (48, 1, 128, 16), (4, 2, 160, 4), (2, 1, 224, 2)])
@pytest.mark.parametrize("kv_lens", [[1], [5, 0, 64, 65], [127, 700, 31, 1, 300]])
def test_single_tokens(hq, hk, dim, page, kv_lens):
    print("case", hq, hk, dim, page, kv_lens, flush=True)
    p = Problem(1 + dim + page + len(kv_lens), [1] * len(kv_lens), kv_lens, hq, hk, dim, page, nhd=page == 16,
                odd=[0, 1, 3][len(kv_lens) % 3])
    p.check(p.run())


@pytest.mark.parametrize("hq,hk,dim,page", [(8, 2, 128, 16), (7, 1, 64, 32), (4, 4, 96, 16), (2, 1, 256, 64), (3, 1, 96, 8),
                                            (2, 2, 192, 1), (5, 1, 32, 16), (2, 1, 160, 16), (3, 1, 224, 4)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([5, 3, 1], [400, 3, 90]), ([0, 2, 0, 9], [10, 2, 0, 333]), ([7], [4]), ([70, 1, 33], [70, 500, 200]),
    ([130], [135]), ([1, 200, 0, 3, 64], [257, 300, 64, 1, 64])])
def test_chunks(hq, hk, dim, page, q_lens, kv_lens):
    print("case", hq, hk, dim, page, q_lens, kv_lens, flush=True)
    p = Problem(7 + dim + sum(q_lens), q_lens, kv_lens, hq, hk, dim, page, nhd=dim == 128, qkv_rows=dim == 64, odd=dim % 3)
    p.check(p.run())


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 10000])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 65]), ([4, 9], [300, 65]), ([66, 1, 5], [190, 129, 40])])
def test_windows(window, q_lens, kv_lens):
    for hq, hk, dim in ((6, 2, 64), (4, 1, 128)):
        print("case", window, q_lens, kv_lens, dim, flush=True)
        p = Problem(window, q_lens, kv_lens, hq, hk, dim, 16)
        p.check(p.run(window=window), window=window)


def test_freed_pages_before_a_window():
    # pages wholly before every window may be gone from the table
    p = Problem(3, [1, 4], [400, 320], 4, 2, 64, 16)
    p.dev[2][0, :(400 - 50) // 16] = -1
    p.dev[2][1, :(320 - 3 - 50) // 16] = -1
    p.check(p.run(window=50), window=50)


@pytest.mark.parametrize("q_len", [1, 40])
def test_long_sequences_split_over_the_chip(q_len):
    for hq, hk, dim, kv in ((4, 1, 128, 9001), (2, 2, 64, 16000)):
        p = Problem(kv + q_len, [q_len, 1], [kv, 77], hq, hk, dim, 32)
        print("case", q_len, kv, flush=True)
        p.check(p.run())


@pytest.mark.parametrize("hq,hk,dim,chunk", [(8, 1, 128, 300), (4, 2, 64, 1100), (2, 1, 256, 600)])
def test_chunks_of_many_rows(hq, hk, dim, chunk):
    # (calls this short have tiles of four waves, of 256 dimensions of eight); rows checked as calls of their own prefix would give them
    kv = chunk + 333
    p = Problem(chunk, [chunk], [kv], hq, hk, dim, 16)
    print("case", hq, hk, dim, chunk, flush=True)
    out, lse = p.run()
    clean = [torch.nan_to_num(t, nan=0.0) for t in (p.k, p.v)]
    for i in (0, 1, 63, chunk // 2, chunk - 2, chunk - 1):
        want = base.ref.attention(p.q[i:i + 1].double(), *clean, p.table.tolist(), [0, 1], [kv - chunk + i + 1], dim ** -0.5)
        tol, lse_tol = base.ref.attention_tolerance(*want, dim)
        assert ((out[i].double() - want[0][0]).abs() <= tol[0]).all()
        assert ((lse[i].double() - want[1][0]).abs() <= lse_tol[0]).all()


@pytest.mark.parametrize("hq,hk,dim", [(32, 8, 128), (24, 4, 64), (8, 2, 96), (20, 2, 32), (16, 8, 256)])
@pytest.mark.parametrize("q_lens,kv_lens", [([5, 1, 6], [1500, 2000, 1030]), ([2] * 20, [1100 + 7 * i for i in range(20)])])
def test_drafted_tokens_of_long_sequences(hq, hk, dim, q_lens, kv_lens):
    # eight waves a work-group up to 192 (sequence, kv head) pairs
    print("case", hq, hk, dim, q_lens, flush=True)
    p = Problem(dim + len(q_lens), q_lens, kv_lens, hq, hk, dim, 16)
    p.check(p.run())
    p.check(p.run(window=400), window=400)


@pytest.mark.parametrize("q_len,seqs,kv", [(1, 64, 20000), (1, 40, 70001), (5, 48, 20011)])
def test_runs_of_many_steps(q_len, seqs, kv):
    # a wave looks pages up for 32 steps at a time; all sequences read the same pages
    p = Problem(q_len, [q_len], [kv], 8, 2, 128, 16)
    single = p.run()
    p.check(single)
    q = p.q_dev.repeat(seqs, 1, 1)
    out, lse = torch.empty_like(q), torch.empty(seqs * q_len, 8, device="cuda")
    ws = torch.zeros(Q.paged_attention_workspace_size(p.cache, seqs * q_len, 8, seqs, q_len, kv), dtype=torch.uint8, device="cuda")
    starts = torch.arange(0, (seqs + 1) * q_len, q_len, dtype=torch.int32, device="cuda")
    lens = torch.full((seqs,), kv, dtype=torch.int32, device="cuda")
    print("case", q_len, seqs, kv, flush=True)
    Q.paged_attention(p.cache, q, out, starts, lens, p.dev[2].expand(seqs, -1).contiguous(), ws, q_len, kv, lse=lse)
    torch.cuda.synchronize()
    for b in range(seqs):
        p.check((out[b * q_len:(b + 1) * q_len].cpu(), lse[b * q_len:(b + 1) * q_len].cpu()))


@pytest.mark.parametrize("q_len", [1, 40])
def test_rows_far_apart(q_len):
    # 2^24 bytes from one row of codes, and of exponent bytes, to the next
    pages, page, dim, hk, kv = 3, 16, 64, 1, 44
    big = [torch.empty(pages, hk, page, 1 << 24, dtype=torch.uint8, device="cuda") for _ in range(4)]
    p = Problem(21, [q_len], [kv], 4, hk, dim, page)
    order = p.dev[2][0].long()
    parts = []
    for t, old, width in zip(big, (p.cache.k, p.cache.v, p.cache.k_scale, p.cache.v_scale), (dim // 2, dim // 2, 2, 2)):
        view = t[..., :width]
        view.copy_(old[order])
        parts.append(view)
    p.cache = Q.KVCache(*parts)
    p.dev[2] = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    got = p.run()
    p.check(got)
    back = [torch.empty(kv, hk, dim, device="cuda") for _ in range(2)]
    Q.kv_read(p.cache, torch.arange(kv, device="cuda"), *back)
    torch.cuda.synchronize()
    for b, t in zip(back, (p.k, p.v)):
        assert torch.equal(b.cpu().double(), t.transpose(1, 2)[order.cpu()].flatten(0, 1)[:kv])


def test_scores_far_apart():
    # scores of some thousands: one key takes all the weight, nothing overflows
    p = Problem(5, [3, 1, 40], [333, 700, 90], 4, 2, 64, 16, magnitude=300.0)
    for scale in (2.0, -2.0, 0.0):
        p.check(p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("q_len,kv,key,window", [(4, 90, 88, 0), (5, 700, 697, 0), (4, 300, 255, 43), (2, 90, 50, 39),
                                                 (60, 190, 150, 0), (60, 190, 140, 33), (600, 700, 650, 0), (70, 70, 69, 0)])
@pytest.mark.parametrize("name", ["k", "v"])
def test_nan_reaches_its_rows_alone(dim, q_len, kv, key, window, name):
    # a block of NaN at a key that only some rows see: those rows get it (of v: in its dimensions), others keep their bits
    p = Problem(31, [q_len], [kv], 4, 2, dim, 16)
    clean = p.run(window=window)
    block = dim // 32 - 1
    p.set_exponent(0, key, block, name, 255 if key % 2 else 253)
    print("case", dim, q_len, kv, key, window, name, flush=True)
    got = p.run(window=window)
    own = kv - q_len + torch.arange(q_len)
    sees = (own >= key) & (own < key + window if window else own >= 0)
    assert sees.any() and not sees.all()
    dims = torch.arange(dim) >= 32 * block if name == "v" else torch.ones(dim, dtype=torch.bool)
    assert torch.isnan(got[0][sees][..., dims].float()).all()
    assert torch.equal(got[0][sees][..., ~dims].view(torch.int16), clean[0][sees][..., ~dims].view(torch.int16))
    assert torch.equal(got[0][~sees].view(torch.int16), clean[0][~sees].view(torch.int16))
    assert torch.equal(got[1][~sees], clean[1][~sees])
    if name == "v":
        assert torch.equal(got[1], clean[1])


@pytest.mark.parametrize("q_len", [1, 4, 40])
def test_nan_that_all_rows_see(q_len):
    for dim in (64, 128, 256):
        for key in (0, 17, 130):
            p = Problem(3, [q_len, 1], [200, 60], 4, 2, dim, 16)
            clean = p.run()
            p.set_exponent(0, key, 1, "v", 254)
            got = p.run()
            assert torch.isnan(got[0][:q_len, :, 32:64].float()).all()
            keep = torch.ones(dim, dtype=torch.bool)
            keep[32:64] = False
            assert torch.equal(got[0][:, :, keep], clean[0][:, :, keep]) and torch.equal(got[0][q_len:], clean[0][q_len:])


def test_a_query_of_nan_stays_in_its_row():
    for q_len in (3, 50):
        p = Problem(2, [q_len], [120], 4, 2, 64, 16)
        clean = p.run()
        p.q_dev[1, 2] = float("nan")
        got = p.run()
        assert torch.isnan(got[0][1, 2].float()).all()
        got[0][1, 2] = clean[0][1, 2]
        assert torch.equal(got[0], clean[0])


def test_lengths_are_cut_to_the_bounds():
    # kv_len past the table or max_kv, and q_start past `tokens`, read nothing beyond
    p = Problem(4, [2, 3], [64, 48], 4, 2, 64, 16)
    full = p.run()
    p.dev[1][0] = 1 << 30
    p.dev[0][2] = 1 << 30
    got = p.run()
    assert torch.equal(got[0], full[0])
    p.dev[1][0] = -5
    got = p.run()
    assert (got[0][:2] == 0).all() and (got[1][:2] == -math.inf).all() and torch.equal(got[0][2:], full[0][2:])


def test_pages_outside_the_cache_count_as_nan():
    for bad in (-1, 1 << 30, -(1 << 31)):
        for q_len in (1, 40):
            p = Problem(4, [q_len, 1], [200, 90], 4, 2, 64, 16)
            full = p.run()
            p.dev[2][0, 3] = bad
            print("case", bad, q_len, flush=True)
            got = p.run()
            assert torch.isnan(got[0][:q_len].float()).all()
            assert torch.equal(got[0][q_len:], full[0][q_len:])


def test_calls_of_all_cache_types_share_a_workspace():
    problems = [Problem(10 + i, [q] * n, [kv] * n, hq, 2, dim, 16) for i, (q, n, kv, hq, dim) in enumerate([
        (1, 2, 3000, 4, 128), (40, 3, 700, 4, 64), (1, 70, 90, 2, 64), (3, 1, 4000, 8, 256), (200, 1, 900, 2, 128),
        (1, 1, 9000, 4, 96), (300, 1, 900, 16, 64)])]
    problems += [base.Problem(40, [1, 1], [3000, 20], 4, 2, 128, 16, "bf16"), base.Problem(41, [70], [900], 4, 2, 64, 16, "e4m3")]
    want = [p.run() for p in problems]
    size = max(Q.paged_attention_workspace_size(p.cache, p.q_start[-1], p.hq, len(p.q_lens), p.max_q, p.max_kv)
               for p in problems)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    order = torch.Generator().manual_seed(0)
    for _ in range(5):
        for i in torch.randperm(len(problems), generator=order).tolist():
            got = problems[i].run(workspace=ws)
            assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1]), i


@pytest.mark.parametrize("seqs", [63, 64, 65, 128, 129, 300, 1100])
@pytest.mark.parametrize("chunks", [0, 1, 2])
def test_many_sequences(seqs, chunks):
    # all in row tiles, as the mean is below 64 rows; single tokens alone, with a few chunks, with long ones
    g = torch.Generator().manual_seed(seqs + chunks)
    q_lens = (torch.rand(seqs, generator=g) < 0.9).int().tolist()
    kv_lens = torch.randint(0, 70, (seqs,), generator=g).tolist()
    for b in range(5, seqs, 60):
        q_lens[b] = [1, 40, 130][chunks]
        kv_lens[b] = q_lens[b] + 25
    q_lens[-1], kv_lens[-1] = q_lens[5], 500
    p = Problem(seqs, q_lens, kv_lens, 4, 2, 64, 16)
    print("case", seqs, chunks, flush=True)
    p.check(p.run())
    if chunks:
        p.check(p.run(window=37), window=37)


@pytest.mark.parametrize("q_len,dim,kv,page", [(1, 64, 60000, 1), (1, 96, 60001, 1), (4, 64, 60013, 1), (40, 64, 30000, 1),
                                               (1, 64, 240000, 2)])
def test_runs_of_more_pages_than_the_list_holds(q_len, dim, kv, page):
    # a work-group's run reaches over more than 1024 pages
    p = Problem(kv + q_len, [q_len], [kv], 1, 1, dim, page)
    print("case", q_len, dim, kv, page, flush=True)
    p.check(p.run(scale=0.5), scale=0.5)


def test_replays_in_a_graph():
    p = Problem(6, [1, 1, 1], [500, 33, 900], 8, 2, 128, 16)
    out = torch.zeros(3, p.hq, p.dim, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(Q.paged_attention_workspace_size(p.cache, 3, p.hq, 3, 1, 900), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    call = lambda: Q.paged_attention(p.cache, p.q_dev, out, *p.dev, ws, 1, 900)
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for lens in ([500, 33, 900], [400, 1, 899], [1, 30, 70]):
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


def test_two_streams_at_once():
    # calls that overlap, each with a workspace of its own
    problems = [Problem(70, [1] * 6, [900, 20, 3000, 1, 77, 512], 8, 2, 128, 16), Problem(71, [300, 2], [700, 4000], 8, 2, 128, 16),
                Problem(72, [4] * 3, [4000, 1500, 90], 16, 2, 64, 16)]
    want = [p.run() for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    spaces = [torch.zeros(Q.paged_attention_workspace_size(p.cache, p.q_start[-1], p.hq, len(p.q_lens), p.max_q, p.max_kv),
                          dtype=torch.uint8, device="cuda") for p in problems]
    outs = [torch.empty(p.q_start[-1], p.hq, p.dim, dtype=torch.bfloat16, device="cuda") for p in problems]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s, w, o in zip(problems, streams, spaces, outs):
            Q.paged_attention(p.cache, p.q_dev, o, *p.dev, w, p.max_q, p.max_kv, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.cpu(), w[0])


def test_offsets_past_32_bits():
    # the last pages of a cache whose codes pass 2^32 bytes, exponent bytes far apart
    hk, page, dim = 8, 128, 128
    pages = (1 << 33) // (hk * page * dim) + 9
    k, v = [torch.zeros(pages, hk, page, dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ke, ve = [torch.zeros(pages, hk, page, 40, dtype=torch.uint8, device="cuda")[..., :4] for _ in range(2)]
    assert ke.stride(0) * (pages - 1) > 1 << 31
    g = torch.Generator().manual_seed(1)
    last = list(range(pages - 3, pages))
    small = []
    for codes, exps in ((k, ke), (v, ve)):
        c, e = mx.encode(torch.randn(3, hk, page, dim, generator=g).double())
        codes[last], exps[last] = c.cuda(), e.cuda()
        small.append(mx.decode(c, e))
    cache = Q.KVCache(k, v, ke, ve)
    for tokens in (1, 40):
        q = torch.randn(tokens, 16, dim, generator=g).bfloat16().cuda()
        out = torch.zeros_like(q)
        table = torch.tensor([last], dtype=torch.int32, device="cuda")
        ws = torch.zeros(Q.paged_attention_workspace_size(cache, tokens, 16, 1, tokens, 300), dtype=torch.uint8, device="cuda")
        Q.paged_attention(cache, q, out, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"),
                          torch.tensor([300], dtype=torch.int32, device="cuda"), table, ws, tokens, 300)
        torch.cuda.synchronize()
        want, lse, spread, slack = base.ref.attention(q.cpu().double(), *small, [[0, 1, 2]], [0, tokens], [300], dim ** -0.5)
        tol, _ = base.ref.attention_tolerance(want, lse, spread, slack, dim)
        assert ((out.cpu().double() - want).abs() <= tol).all()


def test_written_attended_and_read_back():
    """The calls in a row, as a serving step makes them: a prompt and then single
    tokens of three sequences are written, attended to and read back."""
    g = torch.Generator().manual_seed(12)
    hq, hk, dim, page, seqs, room = 8, 2, 128, 16, 3, 96
    cols = room // page
    shape = (seqs * cols, hk, page)
    cache = Q.KVCache(*[torch.zeros(*shape, dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2)],
                      *[torch.zeros(*shape, dim // 32, dtype=torch.uint8, device="cuda") for _ in range(2)])
    rope = Q.Rope(dim, base=500000.0)
    freq, _ = base.ref.rope_frequencies(dim, 500000.0)
    table = torch.randperm(seqs * cols, generator=g).view(seqs, cols)
    lens = [0] * seqs
    size = max(Q.paged_attention_workspace_size(cache, seqs * n, hq, seqs, n, room) for n in (1, 60))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for counts in ([17, 60, 1], [1, 1, 1], [1, 0, 5], [1, 1, 1]):
        total = sum(counts)
        pos = torch.cat([torch.arange(lens[b], lens[b] + n) for b, n in enumerate(counts)])
        slots = torch.cat([table[b][torch.arange(lens[b], lens[b] + n) // page] * page + torch.arange(lens[b], lens[b] + n) % page
                           for b, n in enumerate(counts)])
        x = torch.randn(total, hq + 2 * hk, dim, generator=g)
        dev = x.cuda()
        q, out = [torch.empty(total, hq, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        back = [torch.empty(total, hk, dim, device="cuda") for _ in range(2)]
        lens = [a + n for a, n in zip(lens, counts)]
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        Q.rope_append(cache, rope, dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:], pos.int().cuda(), slots.cuda(), q)
        Q.paged_attention(cache, q, out, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), table.int().cuda(), ws, max(counts), room)
        Q.kv_read(cache, slots.cuda(), *back)
        torch.cuda.synchronize()
        k, _ = base.ref.rotate(x[:, hq:hq + hk].double(), pos, freq, 1.0, dim, False)
        # (positions this small: no rotated key within 2^-40 of a border at this seed)
        for b, want in zip(back, (k, x[:, hq + hk:].double())):
            assert torch.equal(b.cpu().double(), mx.decode(*mx.encode(want)))
        values = [torch.nan_to_num(mx.decode(c.cpu(), e.cpu()), nan=0.0)
                  for c, e in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        want = base.ref.attention(q.cpu().double(), *values, table.tolist(), starts, lens, dim ** -0.5)
        tol, _ = base.ref.attention_tolerance(*want, dim)
        assert ((out.cpu().double() - want[0]).abs() <= tol).all()
