"""Attention over a 4-bit cache by each of its kernels, at the sizes where their
plans change: up to 64, up to 128 and more sequences, rows about a tile.  Which
kernel a call takes goes by its bounds, so every problem here names the one that
it is for, and the library's count of launches has to agree."""
import math

import pytest

from tests.test_parity_gpu_mxfp4_attention import Problem
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROWS, TILES4, TILES8 = "attention_rows", "attention_tiles4", "attention_tiles8"
LOOSE = 1 << 26                 # a max_kv by which no call is a short one


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


def run_by(route, p, **how):
    before = Q.route_count(route)
    got = p.run(**how)
    assert Q.route_count(route) == before + 1, route
    return got


def run_padded(route, p, tokens, window=0, max_kv=LOOSE):
    """A call of `tokens` rows or its own, the ones behind the last sequence's unused: they
    count for the kernel's choice alone, and stay as they were."""
    used = p.q_start[-1]
    tokens = max(tokens, used)
    q = torch.zeros(tokens, p.hq, p.dim, dtype=torch.bfloat16, device="cuda")
    q[:used] = p.q_dev
    out, lse = torch.full_like(q, 7.0), torch.full((tokens, p.hq), 7.0, device="cuda")
    need = Q.paged_attention_workspace_size(p.cache, tokens, p.hq, len(p.q_lens), p.max_q, max_kv)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    before = Q.route_count(route)
    Q.paged_attention(p.cache, q, out, *p.dev, ws, p.max_q, max_kv, window=window, lse=lse)
    torch.cuda.synchronize()
    assert Q.route_count(route) == before + 1, route
    assert (out[used:] == 7.0).all() and (lse[used:] == 7.0).all()
    return out[:used].cpu(), lse[:used].cpu()


def many(seqs, hq, hk, dim, page=16):
    """Single tokens and empty sequences, and longer ones on either side of the
    places where a lane's or the list's sequences end."""
    g = torch.Generator().manual_seed(seqs + dim)
    q_lens = (torch.rand(seqs, generator=g) < 0.9).int().tolist()
    kv_lens = torch.randint(0, 70, (seqs,), generator=g).tolist()
    for b, n in ((5, 300), (62, 20), (63, 33), (64, 17), (126, 9), (127, 40), (128, 35), (seqs - 1, 130)):
        if b < seqs:
            q_lens[b], kv_lens[b] = n, n + 25
    kv_lens[seqs - 1] = 500
    return Problem(seqs, q_lens, kv_lens, hq, hk, dim, page)


@pytest.mark.parametrize("seqs", [63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 1), (160, 16)])
def test_many_sequences_share_tiles(seqs, dim, page):
    # up to 64 and 128 sequences two a lane are planned at once, beyond that threads go through them
    p = many(seqs, 6, 2, dim, page)
    print("case", seqs, dim, flush=True)
    for window in (0, 37):
        p.check(run_by(TILES4, p, window=window), window=window)


@pytest.mark.parametrize("seqs", [1, 64, 65, 128, 129])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_many_sequences_share_tiles_of_eight_waves(seqs, dim):
    p = many(seqs, 6, 1, dim) if seqs > 1 else Problem(3, [400], [500], 6, 1, dim, 16)
    print("case", seqs, dim, flush=True)
    for window in (0, 37):
        p.check(run_padded(TILES8, p, 2048 * seqs // 6 + 1, window=window), window=window)


@pytest.mark.parametrize("group,rows", [(1, 65), (1, 96), (1, 97), (1, 127), (5, 65), (5, 125), (3, 129), (7, 70), (7, 133)])
@pytest.mark.parametrize("window", [0, 1, 17, 64])
def test_rows_about_the_tiles_alone(group, rows, window):
    # one sequence, so that its mean is past 64 rows
    n = -(-rows // group)
    for dim, kv in ((128, n + 700), (64, n)):
        p = Problem(rows + dim, [n], [kv], 2 * group, 2, dim, 16)
        print("case", group, rows, window, dim, flush=True)
        p.check(run_by(ROWS, p, window=window), window=window)
        p.check(run_by(TILES4, p, window=window, max_kv=LOOSE), window=window)
        p.check(run_padded(TILES8, p, 2048 // group + 1, window=window), window=window)


@pytest.mark.parametrize("hq,hk,dim,chunk", [(8, 1, 128, 300), (8, 1, 64, 300), (4, 1, 96, 600)])
def test_chunks_of_many_rows_by_eight_waves(hq, hk, dim, chunk):
    p = Problem(chunk, [chunk], [chunk + 333], hq, hk, dim, 16)
    print("case", hq, hk, dim, chunk, flush=True)
    p.check(run_by(TILES8, p, max_kv=LOOSE))
    p.check(run_by(TILES4, p))


def test_nan_and_lost_pages_among_many_sequences():
    # a NaN block that some rows of the long sequence see, and a page of another outside the cache
    for seqs in (65, 129):
        p = many(seqs, 6, 2, 64)
        runs = [lambda: run_by(TILES4, p), lambda: run_padded(TILES8, p, 2048 * seqs // 3 + 1)]
        clean = [r() for r in runs]
        p.set_exponent(5, 200, 1, "v", 255)
        bad = seqs - 2
        while not (p.q_lens[bad] and p.kv_lens[bad]):
            bad -= 1
        p.dev[2][bad, 0] = -1
        row = p.q_start[bad]
        at = p.q_start[5]
        sees = torch.arange(300) + 25 >= 200
        for r, was in zip(runs, clean):
            got = r()
            assert torch.isnan(got[0][row:row + p.q_lens[bad]].float()).all()
            assert torch.isnan(got[0][at:at + 300][sees][..., 32:].float()).all()
            keep = torch.ones(got[0].shape, dtype=torch.bool)
            keep[row:row + p.q_lens[bad]] = False
            part = keep[at:at + 300]
            part[sees, :, 32:] = False
            assert torch.equal(got[0][keep], was[0][keep])


def test_kernels_share_a_workspace_and_repeat_their_bits():
    calls = [(ROWS, Problem(80, [1] * 40, [700] * 40, 8, 2, 128, 16), {}), (TILES4, many(129, 6, 2, 64), {}),
             (TILES8, Problem(82, [300], [900], 8, 1, 128, 16), {"max_kv": LOOSE}), (ROWS, Problem(83, [40], [900], 4, 2, 64, 16), {}),
             (TILES8, Problem(84, [600], [601], 4, 1, 64, 16), {"max_kv": LOOSE}), (TILES4, Problem(85, [300], [900], 2, 1, 256, 16), {}),
             (TILES8, Problem(86, [300], [900], 4, 1, 256, 16), {"max_kv": LOOSE})]
    want = [run_by(route, p, **how) for route, p, how in calls]
    size = max(Q.paged_attention_workspace_size(p.cache, p.q_start[-1], p.hq, len(p.q_lens), p.max_q, how.get("max_kv", p.max_kv))
               for _, p, how in calls)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    order = torch.Generator().manual_seed(0)
    for _ in range(5):
        for i in torch.randperm(len(calls), generator=order).tolist():
            route, p, how = calls[i]
            got = run_by(route, p, workspace=ws, **how)
            assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1]), i


def test_captured_replays_of_shared_tiles():
    # other lengths at each replay, up to the bounds of the captured call
    for seqs in (65, 129):
        p = many(seqs, 6, 2, 64)
        tokens = p.q_start[-1]
        out = torch.zeros(tokens, p.hq, p.dim, dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(Q.paged_attention_workspace_size(p.cache, tokens, p.hq, seqs, 300, 500), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        call = lambda: Q.paged_attention(p.cache, p.q_dev, out, *p.dev, ws, 300, 500)
        before = Q.route_count(TILES4)
        with torch.cuda.stream(stream):
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        assert Q.route_count(TILES4) == before + 2
        lens = p.kv_lens
        for cut in (0, 7, 24):
            p.kv_lens = [max(0, n - cut) for n in lens]
            p.dev[1].copy_(torch.tensor(p.kv_lens, dtype=torch.int32))
            p.q_dev.mul_(-1.0)
            p.q = p.q_dev.cpu()
            graph.replay()
            torch.cuda.synchronize()
            eager = p.run(workspace=ws, max_kv=500, max_q=300)
            assert torch.equal(out.cpu(), eager[0])
            p.check(eager)
