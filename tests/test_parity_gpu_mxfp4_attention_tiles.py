"""Attention over a 4-bit cache with more rows a sequence and kv head than one
tile holds: in row tiles that each stream the cache, and in the tiles that
waves share.  Which of the two a call takes goes by its bounds: problems here
run once with their own and once with a max_kv far above their lengths, by which
those of 65 to 512 rows and more than 64 in the mean of their sequences change
kernels.  test_parity_gpu_mxfp4_attention_routes.py names the kernel that each
of its problems runs on."""
import math

import pytest

from tests.test_parity_gpu_mxfp4_attention import Problem
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LOOSE = 1 << 26


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


def both(p, **how):
    return [p.run(**how), p.run(max_kv=LOOSE, **how)]


@pytest.mark.parametrize("group", [1, 5, 7])
@pytest.mark.parametrize("rows", [33, 63, 64, 65, 96, 97, 511, 513])
def test_rows_about_the_tiles(group, rows):
    n = -(-rows // group)
    for dim, kv in ((128, n + 700), (64, n)):
        p = Problem(rows + dim, [n, 1], [kv, 90], 2 * group, 2, dim, 16)
        print("case", group, rows, dim, flush=True)
        for got in both(p):
            p.check(got)


@pytest.mark.parametrize("dim,page", [(32, 16), (64, 1), (96, 32), (128, 16), (128, 8), (160, 16), (192, 4), (224, 16), (224, 2),
                                      (256, 64), (256, 1)])
@pytest.mark.parametrize("q_lens,kv_lens", [([24], [24]), ([30, 1, 0, 17, 3], [400, 70, 33, 17, 1000]), ([1, 70], [900, 2100])])
def test_head_dimensions_and_pages(dim, page, q_lens, kv_lens):
    p = Problem(dim + page + len(q_lens), q_lens, kv_lens, 10, 2, dim, page, nhd=page == 16, qkv_rows=dim == 64, odd=dim % 3)
    print("case", dim, page, q_lens, flush=True)
    for got in both(p):
        p.check(got)


@pytest.mark.parametrize("dim,page", [(160, 16), (192, 1), (224, 32), (256, 16), (256, 4)])
@pytest.mark.parametrize("q_lens,kv_lens,window", [([300], [340], 0), ([230, 0, 300], [1000, 20, 300], 0), ([300], [900], 45),
                                                   ([520, 1], [521, 300], 0)])
def test_wide_heads_of_many_rows(dim, page, q_lens, kv_lens, window):
    # past 1024 rows a sequence eight waves share a tile, which read most of their queries from LDS
    p = Problem(dim + page, q_lens, kv_lens, 5, 1, dim, page, nhd=page == 16)
    print("case", dim, page, q_lens, window, flush=True)
    for scale in (0.05, -0.05):
        p.check(p.run(window=window, scale=scale), window=window, scale=scale)


@pytest.mark.parametrize("dim,page", [(32, 16), (64, 16), (64, 1), (96, 8), (128, 16), (128, 64)])
@pytest.mark.parametrize("q_lens,kv_lens,window", [([300], [340], 0), ([600, 0, 500], [1000, 20, 500], 0), ([300], [900], 45),
                                                   ([520, 1], [521, 300], 0)])
def test_eight_waves_to_a_tile(dim, page, q_lens, kv_lens, window):
    # 2048 rows a sequence and more, and a bound by which the call is a long one; with its own four waves
    p = Problem(dim + page, q_lens, kv_lens, 8, 1, dim, page, nhd=page == 16)
    print("case", dim, page, q_lens, window, flush=True)
    for got in both(p, window=window):
        p.check(got, window=window)


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("name", ["k", "v"])
def test_nan_in_a_tile_of_eight_waves(dim, name):
    p = Problem(17, [600], [700], 8, 2, dim, 16)
    clean = both(p)
    p.set_exponent(0, 650, 1, name, 255)
    dims = (torch.arange(dim) // 32 == 1) if name == "v" else torch.ones(dim, dtype=torch.bool)
    for got, was in zip(both(p), clean):
        assert torch.isnan(got[0][550:][..., dims].float()).all()
        assert torch.equal(got[0][550:][..., ~dims], was[0][550:][..., ~dims]) and torch.equal(got[0][:550], was[0][:550])


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 10000])
@pytest.mark.parametrize("q_lens,kv_lens", [([30, 1], [300, 65]), ([44, 9, 0, 1], [45, 65, 0, 700])])
def test_windows(window, q_lens, kv_lens):
    for hq, hk, dim in ((6, 2, 64), (7, 1, 128)):
        p = Problem(window, q_lens, kv_lens, hq, hk, dim, 16)
        print("case", window, q_lens, dim, flush=True)
        for got in both(p, window=window):
            p.check(got, window=window)


def test_freed_pages_before_a_window():
    p = Problem(3, [40, 4], [400, 320], 4, 2, 64, 16)
    p.dev[2][0, :(400 - 39 - 50) // 16] = -1
    p.dev[2][1, :(320 - 3 - 50) // 16] = -1
    for got in both(p, window=50):
        p.check(got, window=50)


@pytest.mark.parametrize("dim,page", [(64, 16), (96, 1), (128, 16), (256, 16)])
@pytest.mark.parametrize("q_len,kv,key,window", [(30, 90, 80, 0), (60, 190, 150, 0), (60, 190, 140, 33), (120, 700, 650, 0),
                                                 (70, 70, 69, 0), (70, 70, 0, 20)])
@pytest.mark.parametrize("name", ["k", "v"])
def test_nan_reaches_its_rows_alone(dim, page, q_len, kv, key, window, name):
    p = Problem(31, [q_len], [kv], 8, 2, dim, page)
    clean = both(p, window=window)
    block = dim // 32 - 1
    p.set_exponent(0, key, block, name, 255 if key % 2 else 253)
    print("case", dim, q_len, kv, key, window, name, flush=True)
    own = kv - q_len + torch.arange(q_len)
    sees = (own >= key) & (own < key + window if window else own >= 0)
    assert sees.any() and not sees.all()
    dims = torch.arange(dim) >= 32 * block if name == "v" else torch.ones(dim, dtype=torch.bool)
    for got, was in zip(both(p, window=window), clean):
        assert torch.isnan(got[0][sees][..., dims].float()).all()
        assert torch.equal(got[0][sees][..., ~dims].view(torch.int16), was[0][sees][..., ~dims].view(torch.int16))
        assert torch.equal(got[0][~sees].view(torch.int16), was[0][~sees].view(torch.int16))
        assert torch.equal(got[1][~sees], was[1][~sees])
        if name == "v":
            assert torch.equal(got[1], was[1])


def test_a_query_of_nan_stays_in_its_row():
    p = Problem(2, [50], [120], 4, 2, 64, 16)
    clean = both(p)
    p.q_dev[33, 2] = float("nan")
    for got, was in zip(both(p), clean):
        assert torch.isnan(got[0][33, 2].float()).all()
        got[0][33, 2] = was[0][33, 2]
        assert torch.equal(got[0], was[0])


def test_lengths_are_cut_to_the_bounds():
    p = Problem(4, [40, 3], [64, 48], 4, 2, 64, 16)
    full = both(p)
    p.dev[1][0] = 1 << 30
    p.dev[0][2] = 1 << 30
    for i, got in enumerate(both(p)):
        assert torch.equal(got[0], full[i][0])
    p.dev[1][0] = -5
    for i, got in enumerate(both(p)):
        assert (got[0][:40] == 0).all() and (got[1][:40] == -math.inf).all() and torch.equal(got[0][40:], full[i][0][40:])


def test_more_tokens_than_the_bound_are_left_alone():
    # a sequence that claims more than max_q tokens is cut to its first max_q rows' tiles
    p = Problem(9, [60, 50], [200, 300], 4, 2, 64, 16)
    out = torch.full((110, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for max_kv in (300, LOOSE):
        ws = torch.zeros(Q.paged_attention_workspace_size(p.cache, 110, 4, 2, 50, max_kv), dtype=torch.uint8, device="cuda")
        out.fill_(7.0)
        Q.paged_attention(p.cache, p.q_dev, out, *p.dev, ws, 50, max_kv)
        got = out.cpu()
        assert (got[50:60] == 7.0).all() and not (got[:50] == 7.0).all(-1).any() and not (got[60:] == 7.0).all(-1).any()


@pytest.mark.parametrize("bad", [-1, 1 << 30, -(1 << 31)])
def test_pages_outside_the_cache_count_as_nan(bad):
    p = Problem(4, [40, 1], [200, 90], 4, 2, 64, 16)
    full = both(p)
    p.dev[2][0, 3] = bad
    for i, got in enumerate(both(p)):
        assert torch.isnan(got[0][:40].float()).all()
        assert torch.equal(got[0][40:], full[i][0][40:])


@pytest.mark.parametrize("seqs", [63, 64, 65, 128, 129, 300, 1100])
@pytest.mark.parametrize("longest", [36, 100])
def test_many_sequences(seqs, longest):
    g = torch.Generator().manual_seed(seqs + longest)
    q_lens = (torch.rand(seqs, generator=g) < 0.9).int().tolist()
    kv_lens = torch.randint(0, 70, (seqs,), generator=g).tolist()
    for b in range(5, seqs, 30):
        q_lens[b] = longest - b % 7
        kv_lens[b] = q_lens[b] + 25
    q_lens[-1], kv_lens[-1] = longest, 500
    p = Problem(seqs, q_lens, kv_lens, 4, 2, 64, 16)
    print("case", seqs, longest, flush=True)
    for window in (0, 37):
        for got in both(p, window=window):
            p.check(got, window=window)


@pytest.mark.parametrize("q_len,hq,dim,kv,page", [(24, 4, 128, 9001, 32), (100, 5, 64, 16000, 16), (40, 2, 64, 30000, 1),
                                                  (70, 1, 96, 20011, 16)])
def test_long_sequences_split_over_the_chip(q_len, hq, dim, kv, page):
    p = Problem(kv + q_len, [q_len, 1], [kv, 77], hq, 1, dim, page)
    print("case", q_len, dim, kv, flush=True)
    for got in both(p):
        p.check(got)


def test_calls_share_a_workspace_and_repeat_their_bits():
    problems = [Problem(50 + i, [q] * n, [kv] * n, hq, 2, dim, 16) for i, (q, n, kv, hq, dim) in enumerate([
        (40, 2, 900, 4, 128), (24, 3, 700, 6, 64), (12, 20, 300, 8, 96), (3, 1, 4000, 8, 256), (200, 1, 900, 2, 128)])]
    want = [both(p) for p in problems]
    ws = torch.zeros(max(Q.paged_attention_workspace_size(p.cache, p.q_start[-1], p.hq, len(p.q_lens), p.max_q, LOOSE)
                         for p in problems), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for p, w in zip(problems, want):
            for got, was in zip(both(p, workspace=ws), w):
                assert torch.equal(got[0], was[0]) and torch.equal(got[1], was[1])


def test_replays_in_a_graph():
    p = Problem(6, [24, 1, 30], [500, 33, 900], 8, 2, 128, 16)
    out = torch.zeros(55, p.hq, p.dim, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(Q.paged_attention_workspace_size(p.cache, 55, p.hq, 3, 30, 900), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    call = lambda: Q.paged_attention(p.cache, p.q_dev, out, *p.dev, ws, 30, 900)
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for starts, lens in (([0, 24, 25, 55], [500, 33, 900]), ([0, 1, 25, 55], [400, 24, 31]), ([0, 25, 54, 55], [30, 29, 70])):
        p.dev[0].copy_(torch.tensor(starts, dtype=torch.int32))
        p.dev[1].copy_(torch.tensor(lens, dtype=torch.int32))
        p.q_start, p.kv_lens = starts, lens
        p.q_lens = [b - a for a, b in zip(starts, starts[1:])]
        p.q_dev.mul_(-1.0)
        p.q = p.q_dev.cpu()
        graph.replay()
        torch.cuda.synchronize()
        eager = p.run(workspace=ws, max_kv=900)
        assert torch.equal(out.cpu(), eager[0])
        p.check(eager)
