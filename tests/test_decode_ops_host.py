"""Host side of the decode operators (no GPU): rotary frequencies against
their definition, and every refusal before anything is enqueued (fake device
addresses that are never read)."""
import ctypes
import math

import numpy as np
import pytest

import tests.decode_reference as ref
from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")

K, V, KS, VS, A, B, C, D, E, F, WS = [(i + 1) << 20 for i in range(11)]
OK, BAD, UNS, ALI = Q.QG_OK, Q.QG_ERR_INVALID_ARG, Q.QG_ERR_UNSUPPORTED, Q.QG_ERR_ALIGNMENT


def _cache(**over):
    vals = dict(k=K, v=V, k_scale=None, v_scale=None, pages=9, page_stride=4 * 16 * 64, head_stride=16 * 64,
                slot_stride=64, kv_heads=4, page_size=16, head_dim=64, dtype=Q.KV_BF16)
    vals.update(over)
    return Q._CacheStruct(**vals)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (40, 10000.0), (128, 1000000.0), (256, 500000.0)])
@pytest.mark.parametrize("opts", [{}, {"scaling": "linear", "factor": 4.0},
                                  {"scaling": "yarn", "factor": 32.0, "original_len": 32768},
                                  {"scaling": "yarn", "factor": 1.0, "original_len": 1, "beta_fast": 4.0, "beta_slow": 0.5}])
def test_rope_frequencies(rot, base, opts):
    rope = Q.Rope(rot, base=base, **opts)
    freq, amp = ref.rope_frequencies(rot, base, opts.get("scaling"), opts.get("factor", 1.0),
                                     opts.get("original_len", 0), opts.get("beta_fast", 32.0), opts.get("beta_slow", 1.0))
    got = np.array([rope._struct.turns[i] for i in range(128)], dtype=np.float64) * 2.0 ** -64 * 2 * math.pi
    # the reference holds 53 bits and pow may be a few of its steps off
    assert np.all(np.abs(got[:rot // 2] - freq) <= 2.0 ** -49 * np.array(freq) + 2.0 ** -62)
    assert not got[rot // 2:].any()
    assert rope._struct.amplitude == np.float32(amp)
    assert Q.Rope(rot, base=base, amplitude=0.5, **opts)._struct.amplitude == 0.5


def test_rope_init_refusals():
    r = Q._RopeStruct()
    good = [8, 0, 10000.0, Q.ROPE_PLAIN, 1.0, 0, 32.0, 1.0, 0.0]
    f = Q.lib().qg_rope_init

    def call(**at):
        args = list(good)
        for i, v in at.items():
            args[int(i[1:])] = v
        return f(ctypes.addressof(r), *args)

    assert call() == OK and f(None, *good) == BAD
    for rot in (0, 1, 7, -2):
        assert call(_0=rot) == BAD
    assert call(_0=258) == UNS and call(_3=3) == UNS and call(_3=-1) == UNS
    for base in (1.0, 0.0, -3.0, math.inf, math.nan):
        assert call(_2=base) == BAD
    for factor in (0.5, 0.0, math.nan, math.inf):
        assert call(_3=Q.ROPE_LINEAR, _4=factor) == BAD
        assert call(_3=Q.ROPE_YARN, _4=factor, _5=100) == BAD
    assert call(_3=Q.ROPE_YARN, _4=2.0, _5=0) == BAD and call(_3=Q.ROPE_YARN, _4=2.0, _5=100) == OK
    for beta in (0.0, -1.0, math.nan, math.inf):
        assert call(_3=Q.ROPE_YARN, _4=2.0, _5=100, _6=beta) == BAD
        assert call(_3=Q.ROPE_YARN, _4=2.0, _5=100, _7=beta) == BAD
    for amp in (-1.0, math.nan, math.inf):
        assert call(_8=amp) == BAD
    with pytest.raises(Q.QGError):
        Q.Rope(8, scaling="other")


CACHE_REFUSALS = [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(pages=0), BAD), (dict(pages=1 << 31), BAD), (dict(kv_heads=0), BAD),
    (dict(page_size=0), BAD), (dict(head_dim=0), BAD), (dict(head_dim=72), UNS), (dict(head_dim=272), UNS),
    (dict(page_size=24, page_stride=4 * 24 * 64), UNS), (dict(page_size=1 << 21), UNS), (dict(dtype=2), UNS),
    (dict(dtype=-1), UNS), (dict(dtype=Q.KV_E4M3), BAD), (dict(dtype=Q.KV_E4M3, k_scale=KS), BAD),
    (dict(slot_stride=56), BAD), (dict(head_stride=0), BAD), (dict(page_stride=8), BAD), (dict(page_stride=-64), BAD),
    (dict(slot_stride=(1 << 31) + 8), BAD), (dict(slot_stride=68), ALI), (dict(head_stride=16 * 64 + 4), ALI),
    (dict(page_stride=4 * 16 * 64 + 2), ALI), (dict(k=K + 8), ALI), (dict(v=V + 2), ALI),
    (dict(dtype=Q.KV_E4M3, k_scale=KS, v_scale=VS, slot_stride=72), ALI),
    (dict(dtype=Q.KV_E4M3, k_scale=KS + 2, v_scale=VS), ALI)]


def _rope_append(cache=None, rope=None, **at):
    args = [A, B, C, Q.SRC_F32, 16 * 64, 64, 16 * 64, 64, 16 * 64, 64, D, E, F, 8 * 64, 64, 3, 8]
    for i, v in at.items():
        args[int(i[1:])] = v
    r = Q.Rope(64) if rope is None else rope
    c = _cache() if cache is None else cache
    return Q.lib().qg_rope_append(ctypes.addressof(c), r._ref, *args, None)


@pytest.mark.parametrize("over,status", CACHE_REFUSALS)
def test_cache_refusals(over, status):
    c = _cache(**over)
    assert _rope_append(cache=c) == status
    assert _attention(cache=c) == status
    assert Q.lib().qg_paged_attention_workspace_size(ctypes.addressof(c), 3, 8, 2, 2, 100) == 0


def test_rope_append_refusals():
    assert _rope_append(_15=0) == OK                     # no tokens: nothing to do
    for i in (0, 1, 2, 10, 11, 12):
        assert _rope_append(**{"_%d" % i: None}) == BAD
    r = Q.Rope(64)
    assert Q.lib().qg_rope_append(None, r._ref, A, B, C, 0, 64, 64, 64, 64, 64, 64, D, E, F, 64, 64, 1, 1, None) == BAD
    assert _rope_append(_15=-1) == BAD and _rope_append(_16=0) == BAD and _rope_append(_15=1 << 31) == BAD
    assert _rope_append(_3=2) == UNS and _rope_append(_16=65536) == UNS
    assert _rope_append(rope=Q.Rope(66)) == BAD          # more than the head has
    for i in range(4, 10):
        assert _rope_append(**{"_%d" % i: -1}) == BAD
    assert _rope_append(_13=63) == BAD and _rope_append(_14=32) == BAD
    for i, off in ((0, 2), (1, 1), (2, 2), (10, 2), (11, 4), (12, 1)):
        assert _rope_append(**{"_%d" % i: A + off}) == ALI


def _attention(cache=None, **at):
    #       q  q strides   out strides     lse       starts lens table strides/cols tokens heads seqs max_q max_kv scale window ws
    args = [A, 8 * 64, 64, B, 8 * 64, 64, None, 8, C, D, E, 7, 7, 3, 8, 2, 2, 100, 0.125, 0, WS, 1 << 30]
    for i, v in at.items():
        args[int(i[1:])] = v
    c = _cache() if cache is None else cache
    return Q.lib().qg_paged_attention(ctypes.addressof(c), *args, None)


def test_attention_refusals():
    for i in (0, 3, 8, 9, 10, 20):
        assert _attention(**{"_%d" % i: None}) == BAD
    for i in (13, 15, 16):                               # nothing to do
        assert _attention(**{"_%d" % i: 0}) == OK
    for i in (12, 13, 15, 16, 17, 19):
        assert _attention(**{"_%d" % i: -1}) == BAD
    for i in (13, 16, 17, 12):
        assert _attention(**{"_%d" % i: 1 << 31}) == BAD
    for heads in (0, -4, 6):
        assert _attention(_14=heads) == BAD
    assert _attention(_15=65536) == UNS
    for scale in (math.nan, math.inf):
        assert _attention(_18=scale) == BAD
    for i in (1, 2, 4, 5, 7, 11):
        assert _attention(_6=F, **{"_%d" % i: -8}) == BAD
    assert _attention(_5=56) == BAD and _attention(_4=32) == BAD and _attention(_6=F, _7=7) == BAD
    for i, off in ((0, 8), (3, 4), (6, 2), (8, 2), (9, 1), (10, 2), (20, 8)):
        assert _attention(**{"_%d" % i: A + off}) == ALI
    assert _attention(_1=8 * 64 + 4) == ALI and _attention(_2=68) == ALI
    assert _attention(_4=8 * 64 + 2) == ALI and _attention(_5=66) == ALI
    c = _cache()
    size = Q.lib().qg_paged_attention_workspace_size(ctypes.addressof(c), 3, 8, 2, 2, 100)
    assert size > 0 and _attention(_21=size - 1) == BAD


def _sample(**at):
    args = [A, 2, 100, 100, B, C, D, E, F, K, WS, 1 << 30]
    for i, v in at.items():
        args[int(i[1:])] = v
    return Q.lib().qg_sample_f32(*args, None)


def test_sample_refusals():
    for i in (0, 4, 9, 10):
        assert _sample(**{"_%d" % i: None}) == BAD
    assert _sample(_1=0) == OK
    for i, vals in ((1, (-1, 65536)), (2, (0, -1, 1 << 31)), (3, (99, -100, (1 << 31) + 1))):
        for v in vals:
            assert _sample(**{"_%d" % i: v}) == BAD
    for i, off in ((0, 2), (4, 1), (5, 2), (6, 2), (7, 1), (8, 2), (9, 2), (10, 8)):
        assert _sample(**{"_%d" % i: A + off}) == ALI
    size = Q.sample_workspace_size(2, 100)
    assert size > 0 and _sample(_11=size - 1) == BAD
    assert Q.sample_workspace_size(-1, 100) == 0 and Q.sample_workspace_size(1, 0) == 0
    assert Q.sample_workspace_size(65536, 10) == 0 and Q.sample_workspace_size(1, 1 << 31) == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(Q.QGError):
        Q.KVCache(k, k)                                                   # not on the GPU
    for bad in (k.float(), k[..., ::2], k[0], k[:0]):
        with pytest.raises(Q.QGError):
            Q.KVCache(bad, bad)
    with pytest.raises(Q.QGError):
        Q.KVCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))    # no scales
    with pytest.raises(Q.QGError):
        Q.KVCache(k, torch.zeros(3, 2, 16, 80, dtype=torch.bfloat16))
    x, u, idx = torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    for args, opts in (((x, u, idx, ws), {}), ((x.double(), u, idx, ws), {}), ((x, u[:1], idx, ws), {}),
                       ((x, u, idx.long(), ws), {}), ((x, u, idx, ws), {"top_k": u}), ((x, u, idx, ws), {"top_p": idx}),
                       ((x.t(), u, idx, ws), {}), ((x[0], u, idx, ws), {})):
        with pytest.raises(Q.QGError):
            Q.sample_f32(*args, **opts)
