"""The 4-bit cache written with rotary positions and read back, on the GPU
against the 64-bit definition.

Codes and exponent bytes have no tolerance where their input is exact (values,
and keys' dimensions that do not turn).  Rotated keys are fp64 in both, off by
some 2^-50 of |x0| + |x1| in either (2^-49 positions of a 53-bit frequency at
2^20 positions: 2^-29): where the definition's element, or the block's largest,
is nearer to a border between two codes (or two scales) than that, either side
of it is right.  Queries: as with the other caches.
"""
import pytest

import tests.decode_reference as ref
import tests.mxfp4_reference as mx
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


def new_cache(g, pages, heads, page, dim, order="phsd", odd=0):
    """Random bytes in a cache of any order of its dimensions; `odd`: exponent
    bytes at odd places, with gaps."""
    sizes = {"p": pages, "h": heads, "s": page, "d": dim}
    out = []
    for each, gap in ((2, 0), (2, 0), (32, odd), (32, odd)):
        shape = [sizes[c] // each if c == "d" else sizes[c] for c in order]
        shape[-1] += gap
        t = torch.randint(0, 250, shape, generator=g, dtype=torch.uint8).cuda()[..., gap:]
        out.append(t.permute([order.index(c) for c in "phsd"]))
    return Q.KVCache(*out)


def rows_of(cache, slots, page):
    """Code and exponent bytes of keys and values at slots, on the CPU: [tokens][heads][...]."""
    where, row = slots // page, slots % page
    return [t.cpu()[where, :, row] for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]


CASES = [
    # tokens, q heads, kv heads, dim, rot, page, source, interleaved, scaling, qkv in one row, order, odd exponents
    (1, 16, 8, 128, 128, 16, "f32", 0, None, 1, "phsd", 0),
    (64, 32, 8, 128, 128, 64, "f32", 0, "yarn", 1, "pshd", 0),
    (7, 4, 4, 64, 32, 16, "bf16", 1, None, 0, "phsd", 1),
    (33, 14, 2, 64, 64, 32, "bf16", 1, "linear", 1, "pshd", 3),
    (5, 8, 8, 96, 40, 16, "bf16", 0, None, 1, "phsd", 0),
    (5, 8, 8, 96, 96, 16, "f32", 1, None, 1, "hpsd", 0),
    (9, 24, 4, 96, 48, 1, "f32", 0, "yarn", 0, "pshd", 1),
    (3, 2, 1, 256, 256, 128, "bf16", 0, None, 1, "phsd", 0),
    (3, 2, 1, 224, 128, 128, "f32", 1, "yarn", 1, "pshd", 0),
    (11, 3, 3, 32, 2, 8, "f32", 0, None, 1, "phsd", 0),
    (11, 3, 1, 160, 6, 8, "bf16", 1, None, 1, "phsd", 5),
    (13, 5, 5, 32, 30, 8, "f32", 0, None, 1, "shpd", 0),
    (300, 40, 8, 128, 64, 16, "bf16", 1, "linear", 1, "phsd", 0),
    (40, 70, 70, 64, 64, 16, "bf16", 0, None, 1, "phsd", 0),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("far", [0, 1])
def test_rope_append(case, far):
    tokens, hq, hk, dim, rot, page, src, inter, scaling, one_row, order, odd = case
    g = torch.Generator().manual_seed(23 * tokens + dim + far)
    pages = -(-tokens // page) + 2
    cache = new_cache(g, pages, hk, page, dim, order, odd)
    before = [t.cpu().clone() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    qkv = torch.randn(tokens, hq + 2 * hk, dim, generator=g) * torch.exp(torch.randn(tokens, hq + 2 * hk, 1, generator=g))
    heads = (qkv if src == "f32" else qkv.bfloat16()).cuda()
    q, k, v = heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:]
    if not one_row:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 4:
        slots[1], slots[4] = -1, pages * page        # both outside the cache
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g) if far else torch.arange(tokens)
    pos[-1] = (1 << 20) - 1 if far else pos[-1]
    opts = {None: {}, "linear": {"scaling": "linear", "factor": 4.0},
            "yarn": {"scaling": "yarn", "factor": 8.0, "original_len": 4096, "amplitude": 1.25}}[scaling]
    rope = Q.Rope(rot, base=500000.0, interleaved=bool(inter), **opts)
    q_out = torch.full((tokens, hq, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    print("case", case, "far", far, flush=True)
    Q.rope_append(cache, rope, q, k, v, pos.int().cuda(), slots.cuda(), q_out)
    torch.cuda.synchronize()
    freq, amp = ref.rope_frequencies(rot, 500000.0, scaling, opts.get("factor", 1.0), opts.get("original_len", 0))
    amp = opts.get("amplitude", amp)
    want, mag = ref.rotate(q.cpu().double(), pos, freq, amp, rot, bool(inter))
    slack = 2.0 ** -20 if not far else 2.0 ** -19
    err = (q_out.cpu().double() - want).abs()
    assert (err <= ref.BF16_HALF * (want.abs() + slack * mag) + slack * mag).all(), float(err.max())

    live = (slots >= 0) & (slots < pages * page)
    at = slots[live]
    got = rows_of(cache, at, page)
    codes, exps = mx.encode(v.cpu().double()[live])
    assert torch.equal(got[2], codes) and torch.equal(got[3], exps)
    want, mag = ref.rotate(k.cpu().double(), pos, freq, amp, rot, bool(inter))
    want, near = want[live], 2.0 ** -28 * mag[live]
    # either side of a border that is as near
    lower, upper = torch.copysign((want.abs() - near).clamp(min=0), want), torch.copysign(want.abs() + near, want)
    options = [mx.encode(x) for x in (want, lower, upper)]
    exact = torch.stack([(got[1] == e) for _, e in options]).any(0)
    assert exact.all()
    nib = lambda t: torch.stack((t & 15, t >> 4), -1).flatten(-2)
    y = want.abs() / torch.pow(torch.tensor(2.0).double(), got[1].double() - 127).repeat_interleave(32, -1)
    nearby = near / torch.pow(torch.tensor(2.0).double(), got[1].double() - 127).repeat_interleave(32, -1)
    size = (nib(got[0]) & 7).long()
    borders = torch.tensor([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1e300], dtype=torch.float64)
    assert ((y >= borders[size] - nearby) & (y <= borders[size + 1] + nearby)).all()
    same = torch.equal(nib(got[0])[near == 0], nib(options[0][0])[near == 0])
    assert same and (nib(got[0]) == nib(options[0][0])).double().mean() > 0.999

    touched = torch.zeros(pages, page, dtype=torch.bool)
    touched[at // page, at % page] = True
    for t, old in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), before):
        keep = ~touched[:, None, :, None].expand(old.shape)
        assert torch.equal(t.cpu()[keep], old[keep])

    # and read back: what the bytes stand for, exactly
    for dtype in (torch.float32, torch.bfloat16):
        back = [torch.full((tokens, hk, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        Q.kv_read(cache, slots.cuda(), *back)
        torch.cuda.synchronize()
        for b, c, e in zip(back, got[0::2], got[1::2]):
            assert torch.equal(b.cpu()[live].double(), mx.decode(c, e))
            assert (b.cpu()[~live] == 7).all()


def test_borders_zeros_and_special_values():
    # values next to every border on either side, the largest and the smallest, infinities and NaN, by the exponent
    g = torch.Generator().manual_seed(2)
    rows = []
    for e in (-140, -126, -125, -30, 0, 3, 100, 124):
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=torch.float64)
        x = torch.cat((mids, mids * (1 + 2.0 ** -23), mids * (1 - 2.0 ** -23), -mids))
        x[0] = 7.0
        rows += [x * 2.0 ** e, x * 2.0 ** e * (1 + 2.0 ** -23)]
    rows.append(torch.zeros(32, dtype=torch.float64))
    rows.append(-torch.zeros(32, dtype=torch.float64))
    for value in (float("inf"), -float("inf"), 3.4e38, -3e38, 1e-45, float("nan")):
        x = torch.randn(32, generator=g).double()
        x[11] = value
        rows.append(x)
    x = torch.stack(rows).float()
    n = x.shape[0]
    cache = new_cache(g, 3, 1, 32, 32)
    src = torch.zeros(n, 3, 32, device="cuda")
    src[:, 1], src[:, 2] = x.cuda(), x.cuda()
    q_out = torch.empty(n, 1, 32, dtype=torch.bfloat16, device="cuda")
    slots = torch.randperm(96, generator=g)[:n]
    Q.rope_append(cache, Q.Rope(32), src[:, :1], src[:, 1:2], src[:, 2:], torch.zeros(n, dtype=torch.int32, device="cuda"),
                  slots.cuda(), q_out)
    torch.cuda.synchronize()
    got = rows_of(cache, slots, 32)
    codes, exps = mx.encode(x.double()[:, None])
    exact = torch.isfinite(x).all(1)                     # (an infinity turns its partner into NaN)
    for i in (0, 2):
        keep = exact if i == 0 else torch.ones_like(exact)
        assert torch.equal(got[i + 1][keep], exps[keep])
        # as numbers: a rotation by 0 of -0 may be +0
        a, b = got[i][keep], codes[keep]
        assert torch.equal(mx.decode(a, got[i + 1][keep]).nan_to_num(nan=9e99), mx.decode(b, exps[keep]).nan_to_num(nan=9e99))


def test_a_long_append_and_read():
    # past 2^23 tokens a call goes in several launches
    tokens, dim = (1 << 23) + 5, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn(1, 3, dim, generator=g, device="cuda").bfloat16()
    src = row.expand(tokens, 3, dim)
    parts = [torch.zeros(2, 1, 16, n, dtype=torch.uint8, device="cuda") for n in (dim // 2, dim // 2, 1, 1)]
    cache = Q.KVCache(*parts)
    slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    slots[0], slots[-1], slots[1 << 23] = 3, 20, 31
    q_out = torch.full((tokens, 1, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    Q.rope_append(cache, Q.Rope(dim), src[:, :1], src[:, 1:2], src[:, 2:], torch.zeros(tokens, dtype=torch.int32, device="cuda"),
                  slots, q_out)
    back = torch.full((tokens, 1, dim), 7.0, device="cuda")
    Q.kv_read(cache, slots, v_out=back)
    torch.cuda.synchronize()
    want = mx.decode(*mx.encode(row[:, 2:].cpu().double()))[0]
    assert (q_out == row[:, :1]).all()
    for t in (0, 1 << 23, tokens - 1):
        assert torch.equal(back[t].cpu().double(), want)
    assert int((back != 7).any(-1).sum()) == 3


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,hk,dim,page,strided", [(1, 1, 32, 1, 0), (3, 8, 128, 16, 0), (70, 2, 96, 4, 1),
                                                        (257, 5, 64, 32, 2), (1000, 3, 256, 128, 0), (41, 300, 32, 8, 1)])
def test_read(kind, dtype, tokens, hk, dim, page, strided):
    g = torch.Generator().manual_seed(tokens + dim)
    pages = -(-tokens // page) + 1
    if kind == "mxfp4":
        cache = new_cache(g, pages, hk, page, dim, "pshd" if strided else "phsd", strided)
        want = [mx.decode(a.cpu(), b.cpu()) for a, b in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    else:
        k, v = torch.randn(2, pages, hk, page, dim, generator=g).to({"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kind])
        k.view(torch.uint8)[0, 0, 0, 0] = 255              # NaN in either type (its low byte in bf16: an ordinary number)
        if kind == "bf16":
            v[0, 0, 0, :8] = torch.tensor([1e-40, -1e-40, float("inf"), -float("inf"), float("nan"), 3e38, -0.0, 1e-38])
            cache = Q.KVCache(k.cuda(), v.cuda())
            want = [k.double(), v.double()]
        else:
            scales = [0.01 + 0.02 * torch.rand(hk, generator=g) for _ in range(2)]
            cache = Q.KVCache(k.cuda(), v.cuda(), *[s.cuda() for s in scales])
            want = [x.float() * s[None, :, None, None] for x, s in zip((k, v), scales)]
    slots = torch.randint(0, pages * page, (tokens,), generator=g)     # some several times
    slots[0] = 0
    if tokens > 2:
        slots[1], slots[2] = -1, pages * page
    if tokens > 40:
        slots[3], slots[4] = -(1 << 63), (1 << 63) - 1
    live = (slots >= 0) & (slots < pages * page)
    outs = []
    for i in range(2):
        wide = torch.full((tokens, hk + 2, dim + (3 if strided == 2 else 8)), 7.0, dtype=dtype, device="cuda")
        outs.append(wide[:, 1:1 + hk, :dim] if strided else wide[:, :hk, :dim].contiguous())
    print("case", kind, dtype, tokens, hk, dim, page, strided, flush=True)
    for which in ((0, 1), (0,), (1,)):
        for o in outs:
            o.fill_(7.0)
        Q.kv_read(cache, slots.cuda(), outs[0] if 0 in which else None, outs[1] if 1 in which else None)
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            got = o.cpu()
            if i not in which:
                assert (got == 7).all()
                continue
            w = want[i].transpose(1, 2).flatten(0, 1)[slots[live]].to(dtype)
            assert torch.equal(got[live].nan_to_num(nan=-77.0), w.nan_to_num(nan=-77.0))
            assert (got[~live] == 7).all()


def test_offsets_past_32_bits():
    # pages past 2^32 bytes of codes and 2^31 bytes of exponents, whose rows are far apart
    hk, page, dim = 8, 128, 256
    pages = (1 << 33) // (hk * page * dim) + 9
    k = torch.zeros(pages, hk, page, dim // 2, dtype=torch.uint8, device="cuda")
    e = torch.full((pages, hk, page, 80), 120, dtype=torch.uint8, device="cuda")[..., :dim // 32]
    cache = Q.KVCache(k, torch.zeros_like(k), e, torch.zeros(pages, hk, page, 80, dtype=torch.uint8, device="cuda")[..., :dim // 32])
    assert e.stride(0) * (pages - 1) > 1 << 31
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 3 * hk, dim, generator=g)
    slots = torch.tensor([(pages - 1) * page + page - 1, (pages - 2) * page])
    src = x.cuda()
    q_out = torch.empty(2, hk, dim, dtype=torch.bfloat16, device="cuda")
    Q.rope_append(cache, Q.Rope(dim), src[:, :hk], src[:, hk:2 * hk], src[:, 2 * hk:],
                  torch.zeros(2, dtype=torch.int32, device="cuda"), slots.cuda(), q_out)
    back = [torch.zeros(2, hk, dim, device="cuda") for _ in range(2)]
    Q.kv_read(cache, slots.cuda(), *back)
    torch.cuda.synchronize()
    for b, part in zip(back, (x[:, hk:2 * hk], x[:, 2 * hk:])):
        assert torch.equal(b.cpu().double(), mx.decode(*mx.encode(part.double())))
    assert int(k[-3:].count_nonzero()) > 0 and int(k[:-3].view(torch.int64).abs().max()) == 0


def test_other_stream_graph_and_torch_types():
    g = torch.Generator().manual_seed(8)
    hq, hk, dim, page, tokens = 4, 2, 64, 16, 5
    k, v = [torch.zeros(3, hk, page, dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ke, ve = [torch.zeros(3, hk, page, dim // 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = Q.KVCache(k.view(torch.float4_e2m1fn_x2), v.view(torch.float4_e2m1fn_x2), ke.view(torch.float8_e8m0fnu),
                      ve.view(torch.float8_e8m0fnu))
    src = torch.randn(tokens, hq + 2 * hk, dim, generator=g).cuda()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    slots = torch.arange(9, 9 + tokens, device="cuda")
    q_out = torch.empty(tokens, hq, dim, dtype=torch.bfloat16, device="cuda")
    back = [torch.empty(tokens, hk, dim, device="cuda") for _ in range(2)]
    rope = Q.Rope(dim)

    def call(stream=None):
        Q.rope_append(cache, rope, src[:, :hq], src[:, hq:hq + hk], src[:, hq + hk:], pos, slots, q_out, stream=stream)
        Q.kv_read(cache, slots, *back, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for step in range(3):
        src.copy_(torch.randn(src.shape, generator=g))
        pos.add_(3)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q_out, *back, k, v, ke, ve)]
        for t in (q_out, *back, k, v, ke, ve):
            t.zero_()
        call()
        torch.cuda.synchronize()
        for a, b in zip(got, (q_out, *back, k, v, ke, ve)):
            assert torch.equal(a, b)
        assert torch.equal(back[1].cpu().double(), mx.decode(*mx.encode(src[:, hq + hk:].cpu().double())))
