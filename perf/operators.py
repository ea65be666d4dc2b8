"""What the decode step's attention block and its token choice are timed on.

Three operators that stand between the library's GEMV calls in a decode or
chunked-prefill step:

  rope    rotary positions on the QKV projection's queries and keys, with the
          keys and values written into a paged cache
  attend  attention of a chunk of new tokens (one token, a few drafted ones or
          thousands) over that cache
  sample  a token per row of LM-head logits, by temperature, top-k, top-p and
          min-p, from given uniform numbers

Each case is a dict of plain values.  With ``own`` false ``run`` computes the
operator from elementary torch operations; with ``own`` true it makes the
library's call.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
VOCAB = 151936            # the LM head of this repository's benchmark


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One user's decode step: a single token after the GEMV, latency only.
        # Heads of the 1024-wide layer (16 query heads, 8 key/value heads).
        _rope("rope_one_token", 1, 16, 8, 128, 128, "f32", "bf16", 16),
        # A serving batch's decode step far into a long context, 8-bit cache.
        _rope("rope_batch64_far_e4m3", 64, 32, 8, 128, 128, "f32", "e4m3", 64, far=1, scaling="yarn", pad=3),
        # A prefill chunk with a partial, interleaved rotation.
        _rope("rope_chunk8191_partial", 8191, 32, 8, 128, 64, "bf16", "bf16", 16, interleaved=1),
        # One user's decode attention over a short context.
        _attend("attend_one_short", 1, 1, 1, 777, 777, 16, 8, 128, "bf16", 16),
        # A serving batch of 32 users whose contexts differ widely.
        _attend("attend_batch32_ragged", 32, 1, 1, 40, 9001, 32, 8, 128, "bf16", 16),
        # Two users with very long contexts in an 8-bit cache.
        _attend("attend_long_e4m3", 2, 1, 1, 120001, 131071, 32, 8, 128, "e4m3", 64, lse=1),
        # Drafted tokens checked in one step (5 per user).
        _attend("attend_draft5", 16, 5, 5, 900, 4099, 16, 8, 128, "bf16", 32),
        # A prefill chunk over what earlier chunks left in the cache.
        _attend("attend_chunk4099", 1, 4099, 4099, 12301, 12301, 32, 8, 128, "bf16", 16),
        # Chunks and single tokens of several users in one call, narrow heads,
        # a sliding window.
        _attend("attend_mixed_window", 24, 1, 777, 1, 6000, 24, 4, 64, "bf16", 32, window=1000),
        # One user's token: the usual top-k and top-p.
        _sample("sample_one", 1, VOCAB, "kp"),
        # A serving batch, each row with settings of its own.
        _sample("sample_batch64", 64, VOCAB, "mix"),
        # Grammar-masked rows, no top-k, a small odd vocabulary.
        _sample("sample_masked", 17, 32001, "pm", masked=1),
    ]


def _rope(name, tokens, q_heads, kv_heads, head_dim, rot_dim, src, kv, page, interleaved=0, far=0, scaling="none",
          pad=0):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot_dim": rot_dim, "src": src, "kv": kv, "page": page,
            "interleaved": bool(interleaved), "far": bool(far), "scaling": scaling, "pad": pad}


def _attend(name, seqs, q_min, q_max, kv_min, kv_max, q_heads, kv_heads, head_dim, kv, page, window=0, lse=0, mix=7):
    return {"name": name, "op": "attend", "seqs": seqs, "q_min": q_min, "q_max": q_max, "kv_min": kv_min,
            "kv_max": kv_max, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "kv": kv,
            "page": page, "window": window, "lse": bool(lse), "mix": mix}


def _sample(name, rows, vocab, kind, masked=0):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "kind": kind, "masked": bool(masked)}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {key: max(work(case)[key] for case in listed()) for key in ("bytes", "flops")}
    while True:
        case = _draw(rng)
        if all(work(case)[key] <= most[key] for key in most):
            return case


def _draw(rng):
    op = rng.choice(["rope", "attend", "attend", "sample"])
    heads, kv_heads = rng.choice([(16, 8), (32, 8), (8, 8), (24, 4), (14, 2), (40, 8)])
    dim = rng.choice([64, 128, 128, 128, 80, 96, 256])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    page = rng.choice([16, 16, 32, 64, 128])
    if op == "rope":
        rot = rng.choice([dim, dim, dim // 2])
        tokens = _log_int(rng, 1, min(8191, 8191 * 48 * 128 // ((heads + 2 * kv_heads) * dim)))
        return _rope(None, tokens, heads, kv_heads, dim, rot, rng.choice(["f32", "bf16"]), kv, page,
                     rng.random() < 0.4, rng.random() < 0.4, rng.choice(["none", "linear", "yarn"]),
                     rng.choice([0, 0, 1]) if tokens > 4 else 0)
    if op == "sample":
        vocab = rng.choice([VOCAB, _log_int(rng, 1000, VOCAB)])
        return _sample(None, _log_int(rng, 1, 64), vocab, rng.choice(["k", "p", "kp", "pm", "mix", "plain"]),
                       rng.random() < 0.3)
    mix = rng.randrange(1 << 20)
    window = rng.choice([0, 0, 0, _log_int(rng, 50, 4000)])
    kind = rng.choice(["decode", "decode", "draft", "chunk", "mixed"])
    if kind == "decode":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 100, 262142 // seqs)
        return _attend(None, seqs, 1, 1, max(1, hi // rng.choice([1, 4, 50])), hi, heads, kv_heads, dim, kv, page,
                       window, rng.random() < 0.5, mix)
    if kind == "draft":
        seqs = _log_int(rng, 1, 32)
        hi = _log_int(rng, 100, 131071 // seqs)
        return _attend(None, seqs, rng.choice([1, 2]), rng.randint(2, 12), max(12, hi // 3), hi, heads, kv_heads, dim,
                       kv, page, window, rng.random() < 0.5, mix)
    if kind == "chunk":
        new = _log_int(rng, 30, 4099)
        total = new + _log_int(rng, 1, 8200)
        return _attend(None, 1, new, new, total, total, heads, kv_heads, dim, kv, page, window, rng.random() < 0.5, mix)
    seqs = rng.randint(2, 24)
    return _attend(None, seqs, 1, _log_int(rng, 20, 777), 1, _log_int(rng, 800, 6000), heads, kv_heads, dim, kv, page,
                   window, rng.random() < 0.5, mix)


# ------------------------------------------------------------- what a case is

def _lengths(case):
    """(new tokens, cached tokens with the new ones) of every sequence: the
    ends of the ranges first, the others between them over their logarithm."""
    rng = random.Random(case["mix"])
    out = []
    for i in range(case["seqs"]):
        new = case["q_max"] if i == 0 else _log_int(rng, case["q_min"], case["q_max"])
        kv = case["kv_max"] if i == 0 else case["kv_min"] if i == 1 else _log_int(rng, case["kv_min"], case["kv_max"])
        out.append((new, max(kv, new)))
    return out


def _pairs_and_keys(new, kv, window):
    """(query, key) pairs that the mask leaves, and keys that some query sees."""
    first = kv - new
    if window <= 0:
        return new * first + new * (new + 1) // 2, kv
    full = max(0, min(new, kv - max(first, window - 1)))   # queries with a whole window
    part = new - full
    return full * window + part * first + part * (part + 1) // 2, kv - max(0, first - window + 1)


def work(case):
    if case["op"] == "rope":
        t, d, hq, hk = case["tokens"], case["head_dim"], case["q_heads"], case["kv_heads"]
        src = 4 if case["src"] == "f32" else 2
        kv = 2 if case["kv"] == "bf16" else 1
        return {"bytes": t * d * ((hq + 2 * hk) * src + hq * 2 + 2 * hk * kv) + t * 12 + case["rot_dim"] * 4,
                "flops": t * (hq + hk) * case["rot_dim"] * 3}
    if case["op"] == "attend":
        d, hq, hk = case["head_dim"], case["q_heads"], case["kv_heads"]
        size = 2 if case["kv"] == "bf16" else 1
        nbytes = flops = 0
        for new, kv in _lengths(case):
            pairs, keys = _pairs_and_keys(new, kv, case["window"])
            nbytes += 2 * keys * hk * d * size + 2 * new * hq * d * 2 + 4 * -(-keys // case["page"])
            nbytes += 4 * new * hq if case["lse"] else 0
            flops += 4 * d * hq * pairs
        return {"bytes": nbytes, "flops": flops}
    return {"bytes": case["rows"] * (case["vocab"] * 4 + 24), "flops": case["rows"] * case["vocab"] * 12}


def _generator(seed, salt):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _cache_dtype(case):
    return torch.bfloat16 if case["kv"] == "bf16" else torch.float8_e4m3fn


def _new_cache(case, g, pages):
    """Keys and values [page][kv head][slot][dim] with what earlier users left
    in them, and each head's scale where the cache is 8-bit."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    k, v = _normal(g, *shape), _normal(g, *shape)
    if case["kv"] == "bf16":
        return k.bfloat16(), v.bfloat16(), None, None
    ks = 0.01 + 0.02 * torch.rand(case["kv_heads"], generator=g, device=DEVICE)
    vs = 0.01 + 0.02 * torch.rand(case["kv_heads"], generator=g, device=DEVICE)
    return ((k / ks[None, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn),
            (v / vs[None, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn), ks, vs)


def _rope_options(case):
    opts = {"rot_dim": case["rot_dim"], "base": 1000000.0, "interleaved": case["interleaved"]}
    if case["scaling"] == "linear":
        opts.update(scaling="linear", factor=4.0)
    elif case["scaling"] == "yarn":
        opts.update(scaling="yarn", factor=32.0, original_len=32768)
    return opts


def _frequencies(case):
    """Angle per position of each rotated pair (64 bits) and the factor on the
    rotated dimensions, from the scaling's definition."""
    rot, base = case["rot_dim"], 1000000.0
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "none":
        return plain, 1.0
    if case["scaling"] == "linear":
        return [f / 4.0 for f in plain], 1.0
    factor, length, fast, slow = 32.0, 32768.0, 32.0, 1.0
    def pair_with(turns):
        return rot * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
    low = max(math.floor(pair_with(fast)), 0)
    high = min(math.ceil(pair_with(slow)), rot - 1)
    out = []
    for i, f in enumerate(plain):
        ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append(f * (1.0 - ramp) + f / factor * ramp)
    return out, 0.1 * math.log(factor) + 1.0


# ---------------------------------------------------------------- prepare

def prepare(case, seed):
    return {"rope": _prepare_rope, "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]](case, seed)


def _prepare_rope(case, seed):
    g = _generator(seed, 11)
    t, d, page = case["tokens"], case["head_dim"], case["page"]
    pages = -(-t // page) + 2
    k_cache, v_cache, ks, vs = _new_cache(case, g, pages)
    # the QKV projection's output: one row per token, queries, keys and values side by side
    width = (case["q_heads"] + 2 * case["kv_heads"]) * d
    qkv = _normal(g, t, width)
    qkv = qkv if case["src"] == "f32" else qkv.bfloat16()
    heads = qkv.view(t, -1, d)
    order = torch.randperm(pages, generator=g, device=DEVICE)
    i = torch.arange(t, device=DEVICE)
    slots = order[i // page] * page + i % page
    if case["pad"]:
        slots[t - case["pad"]:] = -1                    # rows that only fill up the batch
    if t < 256 and case["far"]:
        pos = torch.randint(0, 1 << 20, (t,), generator=g, device=DEVICE)
    else:
        pos = i + ((1 << 20) - t if case["far"] else 333)
    freq, factor = _frequencies(case)
    state = {"case": case, "q": heads[:, :case["q_heads"]],
             "k": heads[:, case["q_heads"]:case["q_heads"] + case["kv_heads"]],
             "v": heads[:, case["q_heads"] + case["kv_heads"]:], "k_cache": k_cache, "v_cache": v_cache,
             "k_scale": ks, "v_scale": vs, "pos": pos.int(), "slots": slots,
             "freq": torch.tensor(freq, dtype=torch.float64, device=DEVICE), "factor": factor,
             "q_out": torch.empty(t, case["q_heads"], d, dtype=torch.bfloat16, device=DEVICE)}
    if own:
        from weight_only_block_amd import qgemv as Q
        state["rope"] = Q.Rope(**_rope_options(case))
        state["cache"] = Q.KVCache(k_cache, v_cache, ks, vs)
    return state


def _prepare_attend(case, seed):
    g = _generator(seed, 22)
    d, page = case["head_dim"], case["page"]
    lengths = _lengths(case)
    need = [-(-kv // page) for _, kv in lengths]
    pages = sum(need) + 3
    k_cache, v_cache, ks, vs = _new_cache(case, g, pages)
    order = torch.randperm(pages, generator=g, device=DEVICE).int()
    table = torch.full((case["seqs"], max(need)), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for new, _ in lengths:
        starts.append(starts[-1] + new)
    q = 2.0 * _normal(g, starts[-1], case["q_heads"], d)
    state = {"case": case, "q": q.bfloat16(), "k_cache": k_cache, "v_cache": v_cache, "k_scale": ks, "v_scale": vs,
             "table": table, "starts": starts, "lengths": lengths, "scale": 1.0 / math.sqrt(d),
             "q_start": torch.tensor(starts, dtype=torch.int32, device=DEVICE),
             "kv_len": torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=DEVICE),
             "out": torch.empty(starts[-1], case["q_heads"], d, dtype=torch.bfloat16, device=DEVICE),
             "lse": torch.empty(starts[-1], case["q_heads"], device=DEVICE) if case["lse"] else None}
    if own:
        from weight_only_block_amd import qgemv as Q
        state["cache"] = Q.KVCache(k_cache, v_cache, ks, vs)
        state["max_q"] = max(new for new, _ in lengths)
        state["max_kv"] = max(kv for _, kv in lengths)
        size = Q.paged_attention_workspace_size(state["cache"], starts[-1], case["q_heads"], case["seqs"],
                                                state["max_q"], state["max_kv"])
        state["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEVICE)
    return state


def _prepare_sample(case, seed):
    g = _generator(seed, 33)
    m, n = case["rows"], case["vocab"]
    # LM-head logits: a broad body and a few tokens that stand out
    logits = 2.5 * _normal(g, m, n)
    hot = torch.randint(0, n, (m, 24), generator=g, device=DEVICE)
    logits.scatter_(1, hot, 9.0 + 3.0 * _normal(g, m, 24))
    if case["masked"]:
        # a grammar leaves about one token in 40, in the first of several rows a single one
        keep = torch.rand(m, n, generator=g, device=DEVICE) < 0.025
        keep.scatter_(1, hot[:, :1], True)
        if m > 4:
            keep[0] = False
            keep[0, n // 2] = True
        logits.masked_fill_(~keep, float("-inf"))
    rnd = random.Random(int(seed) * 77 + 5)
    cols = {"temperature": [], "top_k": [], "top_p": [], "min_p": []}
    for i in range(m):
        kind = rnd.choice(["k", "p", "kp", "pm", "plain", "greedy"]) if case["kind"] == "mix" else case["kind"]
        cols["temperature"].append(0.0 if kind == "greedy" else rnd.choice([0.6, 0.7, 1.0, 1.3]))
        cols["top_k"].append(rnd.choice([20, 50, 1000]) if "k" in kind else 0)
        cols["top_p"].append(rnd.choice([0.8, 0.9, 0.95]) if "p" in kind and kind != "plain" else 1.0)
        cols["min_p"].append(rnd.choice([0.02, 0.05]) if kind == "pm" else 0.0)
    state = {"case": case, "logits": logits, "u": torch.rand(m, generator=g, device=DEVICE),
             "idx": torch.empty(m, dtype=torch.int32, device=DEVICE)}
    for key, vals in cols.items():
        state[key] = torch.tensor(vals, dtype=torch.int32 if key == "top_k" else torch.float32, device=DEVICE)
    if own:
        from weight_only_block_amd import qgemv as Q
        state["workspace"] = torch.zeros(Q.sample_workspace_size(m, n), dtype=torch.uint8, device=DEVICE)
    return state


# -------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if op == "rope":
        return _own_rope(state) if own else _plain_rope(state)
    if op == "attend":
        return _own_attend(state) if own else _plain_attend(state)
    return _own_sample(state) if own else _plain_sample(state)


def _own_rope(s):
    from weight_only_block_amd import qgemv as Q
    Q.rope_append(s["cache"], s["rope"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["q_out"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    from weight_only_block_amd import qgemv as Q
    Q.paged_attention(s["cache"], s["q"], s["out"], s["q_start"], s["kv_len"], s["table"], s["workspace"],
                      s["max_q"], s["max_kv"], scale=s["scale"], window=s["case"]["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]} if s["case"]["lse"] else {"out": s["out"]}


def _own_sample(s):
    from weight_only_block_amd import qgemv as Q
    Q.sample_f32(s["logits"], s["u"], s["idx"], s["workspace"], temperature=s["temperature"], top_k=s["top_k"],
                 top_p=s["top_p"], min_p=s["min_p"])
    return s["idx"]


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y0, y1), -1).flatten(-2) if interleaved else torch.cat((y0, y1), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _to_cache(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x / scale[None, :, None]).clamp(-448, 448).to(dtype)


def _plain_rope(s):
    case = s["case"]
    angle = s["pos"].double()[:, None] * s["freq"][None, :]
    cos = (torch.cos(angle) * s["factor"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["factor"]).float()[:, None, :]
    q = _rotate(s["q"].float(), cos, sin, case["rot_dim"], case["interleaved"])
    k = _rotate(s["k"].float(), cos, sin, case["rot_dim"], case["interleaved"])
    dtype, page = s["k_cache"].dtype, case["page"]
    n = case["tokens"] - case["pad"]
    slots = s["slots"][:n]
    where, row = slots // page, slots % page
    # 8-bit elements are indexed as bytes
    raw = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
    s["k_cache"].view(raw)[where, :, row] = _to_cache(k[:n], s["k_scale"], dtype).view(raw)
    s["v_cache"].view(raw)[where, :, row] = _to_cache(s["v"][:n].float(), s["v_scale"], dtype).view(raw)
    return {"q": q.bfloat16(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, pages, kv, scale):
    """Keys or values of one sequence as [kv head][token][dim] in 32 bits."""
    raw = torch.uint8 if cache.dtype == torch.float8_e4m3fn else cache.dtype
    x = cache.view(raw)[pages].view(cache.dtype).float()
    x = x.permute(1, 0, 2, 3).reshape(cache.shape[1], -1, cache.shape[3])[:, :kv]
    return x if scale is None else x * scale[:, None, None]


def _plain_attend(s):
    case = s["case"]
    hk, d = case["kv_heads"], case["head_dim"]
    group = case["q_heads"] // hk
    outs, lses = [], []
    for b, (new, kv) in enumerate(s["lengths"]):
        pages = s["table"][b, :-(-kv // case["page"])].long()
        k = _gathered(s["k_cache"], pages, kv, s["k_scale"])
        v = _gathered(s["v_cache"], pages, kv, s["v_scale"])
        key = torch.arange(kv, device=DEVICE)
        for lo in range(0, new, 1024):
            hi = min(new, lo + 1024)
            q = s["q"][s["starts"][b] + lo:s["starts"][b] + hi].float()
            q = q.view(hi - lo, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * (hi - lo), d)
            score = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
            score = score.view(hk, group, hi - lo, kv)
            pos = torch.arange(kv - new + lo, kv - new + hi, device=DEVICE)[:, None]
            seen = key <= pos
            if case["window"]:
                seen = seen & (key > pos - case["window"])
            score = score.masked_fill(~seen, float("-inf"))
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - top)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(hk, group * (hi - lo), kv), v).view(hk, group, hi - lo, d) / total
            outs.append(o.permute(2, 0, 1, 3).reshape(hi - lo, hk * group, d).bfloat16())
            lses.append((top + torch.log(total)).squeeze(-1).permute(2, 0, 1).reshape(hi - lo, hk * group))
    out = {"out": torch.cat(outs)}
    if case["lse"]:
        out["lse"] = torch.cat(lses)
    return out


def _plain_sample(s):
    x = s["logits"].double()
    n = x.shape[1]
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"]).double()[:, None]
    top = x.amax(1, keepdim=True)
    w = torch.exp((x - top) / t)
    # most likely first, the lower index first among equals
    _, order = torch.sort(x, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    rank = torch.arange(n, device=DEVICE)[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], n))[:, None]
    keep = rank < k
    ws = ws * keep
    before = torch.cumsum(ws, 1) - ws
    p = s["top_p"].double()[:, None]
    keep = keep & ((before < p * ws.sum(1, keepdim=True)) | (p >= 1) | (rank == 0))
    keep = keep & (ws >= s["min_p"].double().clamp(max=1.0)[:, None])
    kept = torch.zeros_like(w).scatter(1, order, ws * keep)
    cum = torch.cumsum(kept, 1)
    target = s["u"].double()[:, None] * cum[:, -1:]
    pick = (cum <= target).sum(1)
    first = torch.where(x == top, rank, torch.full_like(rank, n)).amin(1)
    return torch.where(greedy, first, pick).int()


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definitions in 64 bits, one sequence or row at a time."""
    state = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](case, state)


def _exact_rope(case, s):
    rot, page = case["rot_dim"], case["page"]
    pairs = [(2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2) for i in range(rot // 2)]
    freq, factor = _frequencies(case)
    first = torch.tensor([a for a, _ in pairs], device=DEVICE)
    second = torch.tensor([b for _, b in pairs], device=DEVICE)
    phase = torch.outer(s["pos"].to(torch.float64), torch.tensor(freq, dtype=torch.float64, device=DEVICE))
    turn = torch.polar(torch.full_like(phase, factor), phase)[:, None, :]

    def turned(x):
        y = x.to(torch.float64).clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": turned(s["q"])}
    for name, new, scale in (("k_cache", turned(s["k"]), s["k_scale"]),
                             ("v_cache", s["v"].to(torch.float64), s["v_scale"])):
        flat = s[name].to(torch.float64).permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["head_dim"])
        if scale is not None:
            new = (new / scale.to(torch.float64)[None, :, None]).clamp(-448.0, 448.0)
        live = s["slots"] >= 0
        flat[s["slots"][live]] = new[live]
        out[name] = flat.view(-1, page, case["kv_heads"], case["head_dim"]).permute(0, 2, 1, 3)
    return out


def _exact_attend(case, s):
    page, group = case["page"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    for b, (new, kv) in enumerate(s["lengths"]):
        ids = s["table"][b].tolist()[:-(-kv // page)]
        at = torch.tensor(ids, device=DEVICE).repeat_interleave(page)[:kv]
        off = torch.arange(kv, device=DEVICE) % page
        for h in range(case["kv_heads"]):
            k = s["k_cache"][:, h].to(torch.float64)[at, off]
            v = s["v_cache"][:, h].to(torch.float64)[at, off]
            if s["k_scale"] is not None:
                k, v = k * float(s["k_scale"][h]), v * float(s["v_scale"][h])
            for lo in range(0, new, 2048):
                hi = min(new, lo + 2048)
                pos = torch.arange(lo, hi, device=DEVICE) + (kv - new)
                far = pos[:, None] - torch.arange(kv, device=DEVICE)[None, :]
                hidden = far < 0
                if case["window"]:
                    hidden |= far >= case["window"]
                for j in range(h * group, (h + 1) * group):
                    rows = slice(s["starts"][b] + lo, s["starts"][b] + hi)
                    logit = (s["q"][rows, j].to(torch.float64) @ k.T) * s["scale"]
                    logit[hidden] = float("-inf")
                    lse[rows, j] = torch.logsumexp(logit, 1)
                    out[rows, j] = torch.softmax(logit, 1) @ v
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_sample(case, s):
    import numpy as np
    logits = s["logits"].cpu().numpy().astype(np.float64)
    vals = {k: s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    picked = []
    for i in range(case["rows"]):
        row = logits[i]
        if vals["temperature"][i] <= 0:
            picked.append(int(np.argmax(row)))
            continue
        order = np.argsort(-row, kind="stable")
        p = np.exp((row[order] - row[order[0]]) / float(vals["temperature"][i]))
        if vals["top_k"][i] > 0:
            order, p = order[:vals["top_k"][i]], p[:vals["top_k"][i]]
        if vals["top_p"][i] < 1:
            ends = np.searchsorted(np.cumsum(p), float(vals["top_p"][i]) * p.sum(), side="left")
            order, p = order[:ends + 1], p[:ends + 1]
        live = p >= min(1.0, float(vals["min_p"][i]))
        order, p = order[live], p[live]
        by_index = np.argsort(order)
        order, p = order[by_index], p[by_index]
        cum = np.cumsum(p)
        j = np.searchsorted(cum, float(vals["u"][i]) * cum[-1], side="right")
        picked.append(int(order[min(j, len(order) - 1)]))
    return torch.tensor(picked, dtype=torch.int32, device=DEVICE)
