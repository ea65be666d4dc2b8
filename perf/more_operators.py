"""What the 4-bit cache's operators are timed on.

A serving process that runs out of memory for keys and values holds them in 4
bits: blocks of 32 dimensions of one token's head, each an exponent byte and 32
codes of one sign, two exponent and one mantissa bit.  Three operators deal
with such a cache:

  write   rotary positions on the QKV projection's queries and keys, keys and
          values quantised into the paged cache, and what the cache now holds
          for these tokens read back (a prefill chunk attends to what later
          tokens will see)
  read    cached tokens read back as bf16 or fp32 rows, for another cache or
          another machine
  attend  attention of new tokens (one, a few drafted ones or thousands) over
          the 4-bit cache

Each case is a dict of plain values.  With ``own`` false ``run`` computes the
operator from elementary torch operations; with ``own`` true it makes the
library's calls.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 32


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One user's decode step: a single token after the GEMV, latency only.
        _write("write_one_token", 1, 16, 8, 128, 128, "f32", 16),
        # A serving batch's decode step far into long contexts, three rows of padding.
        _write("write_batch48_far", 48, 32, 8, 128, 128, "f32", 32, far=1, scaling="yarn", pad=3),
        # A prefill chunk with a partial, interleaved rotation.
        _write("write_chunk6001_partial", 6001, 32, 8, 128, 64, "bf16", 16, interleaved=1),
        # One user's short context handed to another worker.
        _read("read_short", 513, 8, 128, 16, "bf16"),
        # A long shared prefix, read back for a cache of another type.
        _read("read_prefix90001", 90001, 8, 128, 32, "bf16"),
        # Narrow heads, every row at a place of its own, in 32 bits.
        _read("read_scattered_f32", 30011, 4, 64, 16, "f32", scattered=1),
        # One user's decode attention over a short context.
        _attend("attend_one_short", 1, 1, 1, 1023, 1023, 16, 8, 128, 16),
        # A serving batch of 40 users whose contexts differ widely.
        _attend("attend_batch40_ragged", 40, 1, 1, 33, 12007, 32, 8, 128, 16),
        # Three users with very long contexts.
        _attend("attend_long", 3, 1, 1, 110001, 131071, 32, 8, 128, 64, lse=1),
        # Drafted tokens checked in one step (6 per user).
        _attend("attend_draft6", 12, 6, 6, 700, 6007, 32, 8, 128, 32),
        # A prefill chunk over what earlier chunks left in the cache.
        _attend("attend_chunk2503", 1, 2503, 2503, 16007, 16007, 32, 8, 128, 16),
        # Chunks and single tokens of several users in one call, narrow heads,
        # a sliding window.
        _attend("attend_mixed_window", 20, 1, 601, 1, 7001, 24, 4, 64, 32, window=900),
    ]


def _write(name, tokens, q_heads, kv_heads, head_dim, rot_dim, src, page, interleaved=0, far=0, scaling="none", pad=0):
    return {"name": name, "op": "write", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot_dim": rot_dim, "src": src, "page": page, "interleaved": bool(interleaved),
            "far": bool(far), "scaling": scaling, "pad": pad}


def _read(name, tokens, kv_heads, head_dim, page, out, scattered=0):
    return {"name": name, "op": "read", "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "out": out, "scattered": bool(scattered)}


def _attend(name, seqs, q_min, q_max, kv_min, kv_max, q_heads, kv_heads, head_dim, page, window=0, lse=0, mix=5):
    return {"name": name, "op": "attend", "seqs": seqs, "q_min": q_min, "q_max": q_max, "kv_min": kv_min,
            "kv_max": kv_max, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "window": window, "lse": bool(lse), "mix": mix}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {key: max(work(case)[key] for case in listed()) for key in ("bytes", "flops")}
    while True:
        case = _draw(rng)
        if all(work(case)[key] <= most[key] for key in most):
            return case


def _draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    heads, kv_heads = rng.choice([(16, 8), (32, 8), (8, 8), (24, 4), (14, 2), (40, 8)])
    dim = rng.choice([64, 128, 128, 128, 96, 256])
    page = rng.choice([16, 16, 32, 64, 128])
    if op == "write":
        rot = rng.choice([dim, dim, dim // 2])
        return _write(None, _log_int(rng, 1, 8191), heads, kv_heads, dim, rot, rng.choice(["f32", "bf16"]), page,
                      rng.random() < 0.4, rng.random() < 0.4, rng.choice(["none", "linear", "yarn"]), rng.choice([0, 0, 1]))
    if op == "read":
        return _read(None, _log_int(rng, 1, 90001), kv_heads, dim, page, rng.choice(["bf16", "bf16", "f32"]),
                     rng.random() < 0.3)
    mix = rng.randrange(1 << 20)
    window = rng.choice([0, 0, 0, _log_int(rng, 50, 4000)])
    lse = rng.random() < 0.5
    kind = rng.choice(["decode", "decode", "draft", "chunk", "mixed"])
    if kind == "decode":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 100, 393213 // seqs)
        return _attend(None, seqs, 1, 1, max(1, hi // rng.choice([1, 4, 50])), hi, heads, kv_heads, dim, page, window, lse,
                       mix)
    if kind == "draft":
        seqs = _log_int(rng, 1, 32)
        hi = _log_int(rng, 100, 196607 // seqs)
        return _attend(None, seqs, rng.choice([1, 2]), rng.randint(2, 12), max(12, hi // 3), hi, heads, kv_heads, dim,
                       page, window, lse, mix)
    if kind == "chunk":
        new = _log_int(rng, 30, 4001)
        total = new + _log_int(rng, 1, 14000)
        return _attend(None, 1, new, new, total, total, heads, kv_heads, dim, page, window, lse, mix)
    return _attend(None, rng.randint(2, 24), 1, _log_int(rng, 20, 777), 1, _log_int(rng, 800, 7001), heads, kv_heads, dim,
                   page, window, lse, mix)


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
    d, hk = case["head_dim"], case["kv_heads"]
    row = d // 2 + d // BLOCK                               # bytes of a head's keys or values of one token
    if case["op"] == "write":
        t, hq = case["tokens"], case["q_heads"]
        src = 4 if case["src"] == "f32" else 2
        # sources, rotated queries, codes, and the keys and values that the cache now stands for
        return {"bytes": t * ((hq + 2 * hk) * d * src + hq * d * 2 + 2 * hk * row + 2 * hk * d * 2 + 12) + case["rot_dim"] * 4,
                "flops": t * (hq + hk) * case["rot_dim"] * 3 + t * 2 * hk * d * 4}
    if case["op"] == "read":
        t = case["tokens"]
        return {"bytes": t * (2 * hk * (row + d * (2 if case["out"] == "bf16" else 4)) + 8), "flops": t * 2 * hk * d}
    hq = case["q_heads"]
    nbytes = flops = 0
    for new, kv in _lengths(case):
        pairs, keys = _pairs_and_keys(new, kv, case["window"])
        nbytes += 2 * keys * hk * row + 2 * new * hq * d * 2 + 4 * -(-keys // case["page"])
        nbytes += 4 * new * hq if case["lse"] else 0
        flops += 4 * d * hq * pairs
    return {"bytes": nbytes, "flops": flops}


def _generator(seed, salt):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


# ------------------------------------------------- the format, in plain torch

def _encode(x):
    """Rows [..., dim] as code bytes [..., dim / 2] (the even dimension in the
    low four bits) and exponent bytes [..., dim / 32].

    A block's scale is the smallest power of two by which its largest magnitude
    is at most 7, so that no value is off by more than half of the largest step
    (7 to 8 times the scale would be); values round to the nearest of 0, 0.5, 1,
    1.5, 2, 3, 4 and 6 scales, ties to the code that ends in 0."""
    blocks = x.unflatten(-1, (-1, BLOCK))
    mant, exp = torch.frexp(blocks.abs().amax(-1))          # 0.5 <= mant < 1
    e = (exp.int() - 3 + (mant > 0.875).int()).clamp(-125, 125)
    e = torch.where(mant == 0, torch.full_like(e, -125), e)
    y = torch.ldexp(blocks, -e[..., None])
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code | torch.signbit(y).byte() << 3).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).byte()


def _tables():
    levels = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    value = torch.tensor(levels + [-v for v in levels], device=DEVICE)
    scale = torch.tensor([2.0 ** max(-126, b - 127) if b < 255 else math.nan for b in range(256)], device=DEVICE)
    return value, scale


def _decode(codes, exps, tables):
    """Rows in 32 bits, which hold every value exactly."""
    value, scale = tables
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return (value[both].unflatten(-1, (-1, BLOCK)) * scale[exps.long()][..., None]).flatten(-2)


def _new_cache(case, g, pages, filled=True):
    """Codes and exponents of keys and values [page][kv head][slot][...]: keys
    with a magnitude of their own per channel, values of one magnitude."""
    heads, page, dim = case["kv_heads"], case["page"], case["head_dim"]
    if not filled:
        k = torch.randint(0, 256, (2, pages, heads, page, dim // 2), generator=g, device=DEVICE, dtype=torch.uint8)
        e = torch.randint(120, 130, (2, pages, heads, page, dim // BLOCK), generator=g, device=DEVICE, dtype=torch.uint8)
        return {"k": k[0], "v": k[1], "k_exp": e[0], "v_exp": e[1]}
    gain = torch.exp(0.6 * _normal(g, heads, 1, dim))
    k, k_exp = _encode(_normal(g, pages, heads, page, dim) * gain)
    v, v_exp = _encode(_normal(g, pages, heads, page, dim))
    return {"k": k, "v": v, "k_exp": k_exp, "v_exp": v_exp}


def _rope_options(case):
    opts = {"rot_dim": case["rot_dim"], "base": 1000000.0, "interleaved": case["interleaved"]}
    if case["scaling"] == "linear":
        opts.update(scaling="linear", factor=4.0)
    elif case["scaling"] == "yarn":
        opts.update(scaling="yarn", factor=32.0, original_len=32768)
    return opts


def _frequencies(case):
    """Angle per position of each rotated pair (64 bits) and the factor on the
    rotated dimensions, a 32-bit number, from the scaling's definition."""
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
    return out, float(torch.tensor(0.1 * math.log(factor) + 1.0, dtype=torch.float32))


# ---------------------------------------------------------------- prepare

def prepare(case, seed):
    return {"write": _prepare_write, "read": _prepare_read, "attend": _prepare_attend}[case["op"]](case, seed)


def _handle(state):
    """The library's description of the state's cache."""
    from weight_only_block_amd import qgemv as Q
    c = state["cache"]
    state["kv"] = Q.KVCache(c["k"], c["v"], c["k_exp"], c["v_exp"])
    return Q


def _prepare_write(case, seed):
    g = _generator(seed, 11)
    t, d, page = case["tokens"], case["head_dim"], case["page"]
    pages = -(-t // page) + 2
    # the QKV projection's output: one row per token, queries, keys and values side by side
    width = (case["q_heads"] + 2 * case["kv_heads"]) * d
    qkv = _normal(g, t, width)
    qkv = qkv if case["src"] == "f32" else qkv.bfloat16()
    heads = qkv.view(t, -1, d)
    order = torch.randperm(pages, generator=g, device=DEVICE)
    i = torch.arange(t, device=DEVICE)
    slots = order[i // page] * page + i % page
    if case["pad"]:
        slots[t - case["pad"]:] = -1                        # rows that only fill up the batch
    if t < 256 and case["far"]:
        pos = torch.randint(0, 1 << 20, (t,), generator=g, device=DEVICE)
    else:
        pos = i + ((1 << 20) - t if case["far"] else 333)
    freq, factor = _frequencies(case)
    kv = (t, case["kv_heads"], d)
    state = {"case": case, "q": heads[:, :case["q_heads"]],
             "k": heads[:, case["q_heads"]:case["q_heads"] + case["kv_heads"]],
             "v": heads[:, case["q_heads"] + case["kv_heads"]:], "cache": _new_cache(case, g, pages, filled=False),
             "pos": pos.int(), "slots": slots, "freq": torch.tensor(freq, dtype=torch.float64, device=DEVICE),
             "factor": factor, "tables": _tables(),
             "q_out": torch.empty(t, case["q_heads"], d, dtype=torch.bfloat16, device=DEVICE),
             "k_back": torch.zeros(kv, dtype=torch.bfloat16, device=DEVICE),
             "v_back": torch.zeros(kv, dtype=torch.bfloat16, device=DEVICE)}
    if own:
        state["rope"] = _handle(state).Rope(**_rope_options(case))
    return state


def _prepare_read(case, seed):
    g = _generator(seed, 44)
    t, page = case["tokens"], case["page"]
    pages = -(-t // page) + 3
    i = torch.arange(t, device=DEVICE)
    if case["scattered"]:
        slots = torch.randperm(pages * page, generator=g, device=DEVICE)[:t]
    else:
        slots = torch.randperm(pages, generator=g, device=DEVICE)[i // page] * page + i % page
    shape = (t, case["kv_heads"], case["head_dim"])
    dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    state = {"case": case, "cache": _new_cache(case, g, pages), "slots": slots, "tables": _tables(),
             "k_back": torch.empty(shape, dtype=dtype, device=DEVICE), "v_back": torch.empty(shape, dtype=dtype, device=DEVICE)}
    if own:
        _handle(state)
    return state


def _prepare_attend(case, seed):
    g = _generator(seed, 22)
    d, page = case["head_dim"], case["page"]
    lengths = _lengths(case)
    need = [-(-kv // page) for _, kv in lengths]
    pages = sum(need) + 3
    cache = _new_cache(case, g, pages)
    order = torch.randperm(pages, generator=g, device=DEVICE).int()
    table = torch.full((case["seqs"], max(need)), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for new, _ in lengths:
        starts.append(starts[-1] + new)
    q = 1.5 * _normal(g, starts[-1], case["q_heads"], d)
    state = {"case": case, "q": q.bfloat16(), "cache": cache, "tables": _tables(), "table": table, "starts": starts,
             "lengths": lengths, "scale": 1.0 / math.sqrt(d),
             "q_start": torch.tensor(starts, dtype=torch.int32, device=DEVICE),
             "kv_len": torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=DEVICE),
             "out": torch.empty(starts[-1], case["q_heads"], d, dtype=torch.bfloat16, device=DEVICE),
             "lse": torch.empty(starts[-1], case["q_heads"], device=DEVICE) if case["lse"] else None}
    if own:
        Q = _handle(state)
        state["max_q"] = max(new for new, _ in lengths)
        state["max_kv"] = max(kv for _, kv in lengths)
        size = Q.paged_attention_workspace_size(state["kv"], starts[-1], case["q_heads"], case["seqs"], state["max_q"],
                                                state["max_kv"])
        state["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEVICE)
    return state


# -------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if op == "write":
        return _own_write(state) if own else _plain_write(state)
    if op == "read":
        return _own_read(state) if own else _plain_read(state)
    return _own_attend(state) if own else _plain_attend(state)


def _own_write(s):
    from weight_only_block_amd import qgemv as Q
    Q.rope_append(s["kv"], s["rope"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["q_out"])
    Q.kv_read(s["kv"], s["slots"], s["k_back"], s["v_back"])
    return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}


def _own_read(s):
    from weight_only_block_amd import qgemv as Q
    Q.kv_read(s["kv"], s["slots"], s["k_back"], s["v_back"])
    return {"k": s["k_back"], "v": s["v_back"]}


def _own_attend(s):
    from weight_only_block_amd import qgemv as Q
    Q.paged_attention(s["kv"], s["q"], s["out"], s["q_start"], s["kv_len"], s["table"], s["workspace"], s["max_q"],
                      s["max_kv"], scale=s["scale"], window=s["case"]["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]} if s["case"]["lse"] else {"out": s["out"]}


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y0, y1), -1).flatten(-2) if interleaved else torch.cat((y0, y1), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_write(s):
    case, cache, page = s["case"], s["cache"], s["case"]["page"]
    angle = s["pos"].double()[:, None] * s["freq"][None, :]
    cos = (torch.cos(angle) * s["factor"])[:, None, :]
    sin = (torch.sin(angle) * s["factor"])[:, None, :]
    # queries in 32 bits; keys in 64, for their rotated values may lie next to a border between two codes
    q = _rotate(s["q"].float(), cos.float(), sin.float(), case["rot_dim"], case["interleaved"])
    n = case["tokens"] - case["pad"]
    k = _rotate(s["k"][:n].double(), cos[:n], sin[:n], case["rot_dim"], case["interleaved"])
    where, row = s["slots"][:n] // page, s["slots"][:n] % page
    cache["k"][where, :, row], cache["k_exp"][where, :, row] = _encode(k)
    cache["v"][where, :, row], cache["v_exp"][where, :, row] = _encode(s["v"][:n].float())
    s["q_out"].copy_(q)
    s["k_back"][:n] = _decode(cache["k"][where, :, row], cache["k_exp"][where, :, row], s["tables"]).bfloat16()
    s["v_back"][:n] = _decode(cache["v"][where, :, row], cache["v_exp"][where, :, row], s["tables"]).bfloat16()
    return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}


def _plain_read(s):
    cache, page = s["cache"], s["case"]["page"]
    where, row = s["slots"] // page, s["slots"] % page
    s["k_back"].copy_(_decode(cache["k"][where, :, row], cache["k_exp"][where, :, row], s["tables"]))
    s["v_back"].copy_(_decode(cache["v"][where, :, row], cache["v_exp"][where, :, row], s["tables"]))
    return {"k": s["k_back"], "v": s["v_back"]}


def _gathered(codes, exps, pages, kv, tables):
    """Keys or values of one sequence as [kv head][token][dim] in 32 bits."""
    x = _decode(codes[pages], exps[pages], tables)
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :kv]


def _plain_attend(s):
    case, cache = s["case"], s["cache"]
    hk, d = case["kv_heads"], case["head_dim"]
    group = case["q_heads"] // hk
    outs, lses = [], []
    for b, (new, kv) in enumerate(s["lengths"]):
        pages = s["table"][b, :-(-kv // case["page"])].long()
        k = _gathered(cache["k"], cache["k_exp"], pages, kv, s["tables"])
        v = _gathered(cache["v"], cache["v_exp"], pages, kv, s["tables"])
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


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definitions in 64 bits, one sequence or head at a time."""
    state = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, state)


def _exact_value(codes, exps):
    """What code bytes [..., dim / 2] and exponent bytes [..., dim / 32] stand for."""
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    for half, nibble in ((0, codes % 16), (1, codes // 16)):
        size, sign = (nibble % 8).to(torch.float64), 1.0 - 2.0 * (nibble // 8).to(torch.float64)
        top, low = torch.div(size, 2, rounding_mode="floor"), size % 2
        out[..., half::2] = sign * torch.where(top == 0, low / 2, (1 + low / 2) * 2.0 ** (top - 1))
    power = torch.pow(2.0, exps.to(torch.float64) - 127.0)
    return out * power.repeat_interleave(BLOCK, -1)


def _exact_rounded(x):
    """Values in 64 bits rounded to the format's."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    most = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(most.clamp(min=1e-300))) - 2
    e = torch.where(torch.pow(2.0, e) * 8 <= most, e + 1, torch.where(torch.pow(2.0, e) * 4 > most, e - 1, e))
    scale = torch.pow(2.0, torch.where(most > 7 * torch.pow(2.0, e), e + 1, e).clamp(-125, 125))
    y = (b / scale).abs()
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).to(torch.float64)
    return (torch.copysign((torch.round(y / step) * step).clamp(max=6.0), b) * scale).reshape(x.shape)


def _exact_write(case, s):
    rot = case["rot_dim"]
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

    live = (s["slots"] >= 0)[:, None, None]
    zero = torch.zeros((), dtype=torch.float64, device=DEVICE)
    return {"q": turned(s["q"]), "k": torch.where(live, _exact_rounded(turned(s["k"])), zero),
            "v": torch.where(live, _exact_rounded(s["v"].to(torch.float64)), zero)}


def _exact_read(case, s):
    out = {}
    for name in ("k", "v"):
        codes, exps = (s["cache"][n].transpose(1, 2).flatten(0, 1)[s["slots"]] for n in (name, name + "_exp"))
        out[name] = _exact_value(codes, exps)
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
            k, v = (_exact_value(s["cache"][n][:, h][at, off], s["cache"][n + "_exp"][:, h][at, off]) for n in ("k", "v"))
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
