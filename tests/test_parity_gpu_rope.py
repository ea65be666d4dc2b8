"""Rotary positions with cache append on the GPU against the 64-bit definition.

Tolerances: the angle reaches fp32 within half a turn (2^-24 relative, at most
2e-7 radians), cos and sin are fp32 functions of it (2^-22 together with the
amplitude's product) and the rotation adds three fp32 roundings: 2^-20 of
|x0| + |x1| covers them.  Then one rounding to the output's type, at most half
a step.
"""
import pytest

import tests.decode_reference as ref
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _require_gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    Q.lib()


def _cache(g, pages, heads, page, dim, kind, nhd=False):
    shape = (pages, page, heads, dim) if nhd else (pages, heads, page, dim)
    k, v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
    if nhd:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    if kind == "bf16":
        return Q.KVCache(k.bfloat16().cuda(), v.bfloat16().cuda())
    ks, vs = 0.01 + 0.02 * torch.rand(heads, generator=g), 0.01 + 0.02 * torch.rand(heads, generator=g)
    return Q.KVCache((10 * k).to(torch.float8_e4m3fn).cuda(), (10 * v).to(torch.float8_e4m3fn).cuda(), ks.cuda(), vs.cuda())


def _bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


CASES = [
    # tokens, q heads, kv heads, dim, rot, page, source, cache, interleaved, scaling, qkv in one row, slots first
    (1, 16, 8, 128, 128, 16, "f32", "bf16", 0, None, 1, 0),
    (64, 32, 8, 128, 128, 64, "f32", "e4m3", 0, "yarn", 1, 1),
    (7, 4, 4, 64, 32, 16, "bf16", "bf16", 1, None, 0, 0),
    (33, 14, 2, 64, 64, 32, "bf16", "e4m3", 1, "linear", 1, 1),
    (5, 8, 8, 80, 40, 16, "bf16", "bf16", 0, None, 1, 0),
    (5, 8, 8, 80, 40, 16, "f32", "e4m3", 1, None, 1, 0),
    (9, 24, 4, 96, 96, 1, "f32", "bf16", 0, "yarn", 0, 1),
    (3, 2, 1, 256, 256, 128, "bf16", "bf16", 0, None, 1, 0),
    (3, 2, 1, 256, 128, 128, "f32", "e4m3", 1, "yarn", 1, 1),
    (11, 3, 3, 16, 2, 8, "f32", "bf16", 0, None, 1, 0),
    (11, 3, 1, 48, 6, 8, "bf16", "e4m3", 1, None, 1, 0),
    (300, 40, 8, 128, 64, 16, "bf16", "bf16", 1, "linear", 1, 0),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("far", [0, 1])
def test_rope_append(case, far):
    tokens, hq, hk, dim, rot, page, src, kind, inter, scaling, one_row, nhd = case
    g = torch.Generator().manual_seed(17 * tokens + dim + far)
    pages = -(-tokens // page) + 2
    cache = _cache(g, pages, hk, page, dim, kind, bool(nhd))
    before_k, before_v = cache.k.cpu().clone(), cache.v.cpu().clone()
    width = (hq + 2 * hk) * dim
    qkv = torch.randn(tokens, width, generator=g)
    qkv = qkv if src == "f32" else qkv.bfloat16()
    heads = qkv.cuda().view(tokens, -1, dim)
    q, k, v = heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:]
    if not one_row:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 4:
        slots[1], slots[4] = -1, pages * page        # both outside the cache
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g) if far else torch.arange(tokens)
    pos[-1] = (1 << 31) - 1 if far else pos[-1]
    opts = {None: {}, "linear": {"scaling": "linear", "factor": 4.0},
            "yarn": {"scaling": "yarn", "factor": 8.0, "original_len": 4096}}[scaling]
    rope = Q.Rope(rot, base=500000.0, interleaved=bool(inter), **opts)
    q_out = torch.full((tokens, hq, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    print("case", case, "far", far, flush=True)
    Q.rope_append(cache, rope, q, k, v, pos.int().cuda(), slots.cuda(), q_out)
    torch.cuda.synchronize()
    freq, amp = ref.rope_frequencies(rot, 500000.0, scaling, opts.get("factor", 1.0), opts.get("original_len", 0))
    want, mag = ref.rotate(q.cpu().double(), pos, freq, amp, rot, bool(inter))
    # 2^31 positions of a 53-bit frequency reach 2^-21 radians in the reference itself
    slack = 2.0 ** -20 if not far else 2.0 ** -19
    err = (q_out.cpu().double() - want).abs()
    assert (err <= ref.BF16_HALF * (want.abs() + slack * mag) + slack * mag).all(), float(err.max())

    want_k, mag_k = ref.rotate(k.cpu().double(), pos, freq, amp, rot, bool(inter))
    got_k, got_v = cache.k.cpu(), cache.v.cpu()
    live = [t for t in range(tokens) if 0 <= int(slots[t]) < pages * page]
    touched = torch.zeros(pages, page, dtype=torch.bool)
    for t in live:
        pg, row = int(slots[t]) // page, int(slots[t]) % page
        touched[pg, row] = True
        x, value = want_k[t], v[t].cpu().float()
        if kind == "bf16":
            err = (got_k[pg, :, row].double() - x).abs()
            assert (err <= ref.BF16_HALF * (x.abs() + slack * mag_k[t]) + slack * mag_k[t]).all()
            assert torch.equal(_bits(got_v[pg, :, row].contiguous()), _bits(value.bfloat16()))
        else:
            ks, vs = cache.k_scale.cpu()[:, None], cache.v_scale.cpu()[:, None]
            y = (x / ks.double()).clamp(-448, 448)
            m = slack * mag_k[t] / ks.double() + 2.0 ** -23 * y.abs()
            err = (got_k[pg, :, row].float().double() - y).abs()
            assert (err <= torch.maximum(ref.E4M3_HALF * (y.abs() + m), torch.tensor(ref.E4M3_TINY)) + m).all()
            want_v = (value / vs).clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(_bits(got_v[pg, :, row].contiguous()), _bits(want_v))
    keep = ~touched[:, None, :, None].expand(pages, hk, page, dim)
    assert torch.equal(_bits(got_k)[keep], _bits(before_k)[keep])
    assert torch.equal(_bits(got_v)[keep], _bits(before_v)[keep])


def test_special_values_reach_the_cache():
    # infinities clamp to the largest code, NaN stays one, in both cache types
    x = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30, -1e30, 0.0, -0.0, 1.0] * 2)
    for kind in ("bf16", "e4m3"):
        g = torch.Generator().manual_seed(3)
        cache = _cache(g, 2, 1, 4, 16, kind)
        src = torch.zeros(1, 3, 16, device="cuda")
        src[0, 2] = x.cuda()
        q_out = torch.empty(1, 1, 16, dtype=torch.bfloat16, device="cuda")
        Q.rope_append(cache, Q.Rope(16), src[:, :1], src[:, 1:2], src[:, 2:], torch.zeros(1, dtype=torch.int32, device="cuda"),
                      torch.tensor([5], device="cuda"), q_out)
        got = cache.v.cpu()[1, 0, 1].float()
        want = x.bfloat16().float() if kind == "bf16" else \
            (x / cache.v_scale.cpu()).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert torch.equal(got[ok], want[ok])
        assert (q_out == 0).all()


def test_unaligned_rows_and_other_stream():
    # rows that start between 16-byte places take the narrow path, on a stream of the caller's
    g = torch.Generator().manual_seed(5)
    tokens, dim = 6, 64
    base = torch.randn(tokens, 3 * dim + 3, generator=g).cuda()
    rows = [base[:, 1 + i * dim:1 + (i + 1) * dim].unsqueeze(1) for i in range(3)]
    outs = []
    for aligned in (0, 1):
        cache = _cache(torch.Generator().manual_seed(6), 2, 1, 8, dim, "bf16")
        q_out = torch.empty(tokens, 1, dim, dtype=torch.bfloat16, device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        x = [r.contiguous() for r in rows] if aligned else rows
        pos = torch.arange(100, 100 + tokens, dtype=torch.int32, device="cuda")
        slots = torch.arange(3, 3 + tokens, device="cuda")
        stream.wait_stream(torch.cuda.current_stream())
        Q.rope_append(cache, Q.Rope(dim), x[0], x[1], x[2], pos, slots, q_out, stream=stream)
        stream.synchronize()
        outs.append((q_out.cpu(), cache.k.cpu(), cache.v.cpu()))
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
