"""Host side of the 4-bit cache (no GPU): the format's reference against its
definition, and every refusal before anything is enqueued (fake device
addresses that are never read)."""
import ctypes
import itertools

import pytest

import tests.mxfp4_reference as mx
from tests.test_decode_ops_host import (ALI, BAD, OK, UNS, A, B, C, _attention, _cache, _rope_append)
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")

KB, VB = 20 << 20, 21 << 20


def _mxfp4(**over):
    vals = dict(dtype=Q.KV_MXFP4, k_block_scale=KB, v_block_scale=VB, scale_page_stride=4 * 16 * 2,
                scale_head_stride=16 * 2, scale_slot_stride=2)
    vals.update(over)
    return _cache(**vals)


def test_reference_format():
    # each element against a search over all levels; the scale against a search over all powers of two
    g = torch.Generator().manual_seed(0)
    x = torch.randn(200, 64, generator=g, dtype=torch.float64) * torch.exp(4 * torch.randn(200, 1, generator=g, dtype=torch.float64))
    x[0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.9, 0.0, -0.0, -0.25, -0.75, -1.25, -2.5, -5.0, 7.0])
    x[0, 16:32] = 7.0
    x[1, :32] = 0.0
    x[2, 5] = float("nan")
    codes, exps = mx.encode(x)
    y = mx.decode(codes, exps)
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64), exps.double() - 127).repeat_interleave(32, -1)
    assert torch.isnan(y[2, :32]).all() and not torch.isnan(y[2, 32:]).any() and exps[2, 0] == 255
    fine = ~torch.isnan(y)
    levels = torch.tensor(mx.LEVELS, dtype=torch.float64)
    best = (x[..., None].abs() - levels * scale[..., None]).abs().amin(-1)
    assert torch.equal((x - y).abs()[fine], best[fine]) and ((x - y).abs()[fine] <= scale[fine]).all()
    assert y[0, :7].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0] and exps[0, 0] == 127
    most = x.reshape(200, 2, 32).abs().amax(-1)
    s = scale[:, ::32]
    live = (most > 0) & ~torch.isnan(most)
    assert (most[live] <= 7 * s[live]).all() and (most[live] > 3.5 * s[live]).all()


MX_REFUSALS = [
    (dict(k_block_scale=None), BAD), (dict(v_block_scale=None), BAD), (dict(head_dim=80), UNS), (dict(head_dim=48), UNS),
    (dict(head_dim=272), UNS), (dict(dtype=2), UNS), (dict(dtype=4), UNS), (dict(slot_stride=72), ALI),
    (dict(slot_stride=80), ALI), (dict(head_stride=16 * 64 + 16), ALI), (dict(k=A + 8), ALI), (dict(slot_stride=32), BAD),
    (dict(scale_slot_stride=1), BAD), (dict(scale_slot_stride=-2), BAD), (dict(scale_head_stride=30), BAD),
    (dict(scale_page_stride=(1 << 31) + 1), BAD), (dict(scale_page_stride=0), BAD)]


def _read(cache=None, **at):
    #       slots k  v  dtype        k strides    v strides   tokens
    args = [A, B, C, Q.SRC_BF16, 4 * 64, 64, 4 * 64, 64, 3]
    for i, v in at.items():
        args[int(i[1:])] = v
    c = _mxfp4() if cache is None else cache
    return Q.lib().qg_kv_read(ctypes.addressof(c), *args, None)


@pytest.mark.parametrize("over,status", MX_REFUSALS)
def test_cache_refusals(over, status):
    c = _mxfp4(**over)
    assert _rope_append(cache=c) == status and _attention(cache=c) == status and _read(cache=c) == status
    assert Q.lib().qg_paged_attention_workspace_size(ctypes.addressof(c), 3, 8, 2, 2, 100) == 0


def test_what_the_other_calls_refuse():
    c = _mxfp4()
    assert _rope_append(cache=c, _15=0) == OK and _attention(cache=c, _13=0) == OK
    # exponent bytes of any alignment and order
    for over in (dict(k_block_scale=KB + 1), dict(scale_slot_stride=3, scale_head_stride=48, scale_page_stride=192 + 1),
                 dict(scale_page_stride=2, scale_head_stride=18, scale_slot_stride=72)):
        assert _rope_append(cache=_mxfp4(**over), _15=0) == OK, over
    size = Q.lib().qg_paged_attention_workspace_size(ctypes.addressof(c), 3, 8, 2, 2, 100)
    assert size > 0 and _attention(cache=c, _21=size - 1) == BAD


def test_read_refusals():
    assert Q.lib().qg_kv_read(None, A, B, C, 0, 64, 64, 64, 64, 1, None) == BAD
    for c in (_mxfp4(), _cache(), _cache(dtype=Q.KV_E4M3, k_scale=KB, v_scale=VB)):
        assert _read(cache=c, _8=0) == OK
        assert _read(cache=c, _0=None) == BAD and _read(cache=c, _1=None, _2=None) == BAD
        assert _read(cache=c, _3=2) == UNS and _read(cache=c, _3=-1) == UNS
        assert _read(cache=c, _8=-1) == BAD and _read(cache=c, _8=1 << 31) == BAD
        for i in (4, 5, 6, 7):
            assert _read(cache=c, **{"_%d" % i: -1}) == BAD and _read(cache=c, **{"_%d" % i: (1 << 31) + 1}) == BAD
            assert _read(cache=c, **{"_%d" % i: 63}) == BAD       # rows that overlap
        for i, off in ((0, 4), (1, 1), (2, 1)):
            assert _read(cache=c, **{"_%d" % i: A + off}) == ALI
        assert _read(cache=c, _1=B + 2, _3=Q.SRC_F32) == ALI
    # what is not wanted is not looked at
    assert _read(_1=None, _4=-1, _5=-1, _8=0) == OK and _read(_2=None, _6=-1, _7=-1, _8=0) == OK


@pytest.mark.parametrize("hq,hk", [(8, 1), (16, 8), (48, 1)])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 256])
def test_an_attention_workspace_serves_smaller_calls(hq, hk, dim):
    c = _mxfp4(kv_heads=hk, head_dim=dim, pages=1 << 20, page_stride=hk * 16 * dim, head_stride=16 * dim, slot_stride=dim,
               scale_page_stride=hk * 16 * (dim // 32), scale_head_stride=16 * (dim // 32), scale_slot_stride=dim // 32)
    ref, fn = ctypes.addressof(c), Q.lib().qg_paged_attention_workspace_size
    tokens, seqs, max_q, max_kv = [1, 31, 302, 2048, 9000], [1, 2, 40, 300], [1, 5, 33, 302, 9000], [1, 100, 5000, 1 << 20]
    size = {s: fn(ref, s[0], hq, s[1], s[2], s[3]) for s in itertools.product(tokens, seqs, max_q, max_kv)}
    assert min(size.values()) > 0
    for a, b in itertools.product(size, size):
        if all(x <= y for x, y in zip(a, b)):
            assert size[a] <= size[b], (a, b)


def test_binding_refuses_host_tensors_types_and_shapes():
    k, e = torch.zeros(3, 2, 16, 32, dtype=torch.uint8), torch.zeros(3, 2, 16, 2, dtype=torch.uint8)
    for args in ((k, k, e, e),                                           # not on the GPU
                 (k, k), (k, k, e), (k, k, e.float(), e.float()), (k, k, e[..., :1], e[..., :1]),
                 (k, k, e, e.transpose(0, 1).contiguous().transpose(0, 1)), (k, k.bfloat16(), e, e),
                 (k[..., :24], k[..., :24], e, e), (k, k, e.repeat(1, 1, 1, 2)[..., ::2], e.repeat(1, 1, 1, 2)[..., ::2])):
        with pytest.raises(Q.QGError):
            Q.KVCache(*args)
