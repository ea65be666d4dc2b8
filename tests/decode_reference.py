"""64-bit definitions of the decode operators, on the CPU, for their tests."""
import math

import numpy as np
import torch

BF16_HALF = 2.0 ** -8        # half a step of a bf16 value, relative
E4M3_HALF = 2.0 ** -4
E4M3_TINY = 2.0 ** -10       # half of the 8-bit format's smallest step


def rope_frequencies(rot, base, scaling=None, factor=1.0, original_len=0, fast=32.0, slow=1.0):
    """f_i per pair and the amplitude, from the scaling's definition."""
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling in (None, "none"):
        return plain, 1.0
    if scaling == "linear":
        return [f / factor for f in plain], 1.0

    def pair_with(turns):
        return rot * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

    low = max(math.floor(pair_with(fast)), 0)
    high = min(math.ceil(pair_with(slow)), rot - 1)
    out = []
    for i, f in enumerate(plain):
        ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append(f * (1.0 - ramp) + f / factor * ramp)
    return out, 0.1 * math.log(factor) + 1.0


def rotate(x, pos, freq, amplitude, rot, interleaved):
    """x [tokens][heads][dim] float64, pos [tokens] -> (rotated, sum of the
    magnitudes that make up each rotated element)."""
    angle = torch.outer(pos.double(), torch.tensor(freq, dtype=torch.float64))
    cos, sin = (torch.cos(angle) * amplitude)[:, None, :], (torch.sin(angle) * amplitude)[:, None, :]
    y, mag = x.clone(), torch.zeros_like(x)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    mag[..., a] = mag[..., b] = amplitude * (x[..., a].abs() + x[..., b].abs())
    return y, mag


def attention(q, k_cache, v_cache, table, q_start, kv_len, scale, window=0, k_scale=None, v_scale=None):
    """q [tokens][heads][dim] and caches as float64, table and lengths as
    lists.  Returns out, lse, spread = softmax-weighted |v| and slack = the
    largest sum of |q k| terms of each row, times |scale| (both for the
    tolerances).  Rows that see nothing: 0 and -inf."""
    tokens, heads, dim = q.shape
    kv_heads, page = k_cache.shape[1], k_cache.shape[2]
    group = heads // kv_heads
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    slack = torch.zeros(tokens, heads, dtype=torch.float64)
    for b, kv in enumerate(kv_len):
        q0, q1 = q_start[b], q_start[b + 1]
        if q1 <= q0 or kv <= 0:
            continue
        at = [(table[b][j // page], j % page) for j in range(kv)]
        pages = torch.tensor([p for p, _ in at])
        rows = torch.tensor([r for _, r in at])
        for h in range(kv_heads):
            k, v = k_cache[pages, h, rows], v_cache[pages, h, rows]
            if k_scale is not None:
                k, v = k * float(k_scale[h]), v * float(v_scale[h])
            for i in range(q1 - q0):
                own = kv - (q1 - q0) + i
                lo = max(0, own - window + 1) if window > 0 else 0
                if own < lo:
                    continue
                for g in range(h * group, (h + 1) * group):
                    x = q[q0 + i, g]
                    s = (k[lo:own + 1] @ x) * scale
                    p = torch.softmax(s, 0)
                    out[q0 + i, g] = p @ v[lo:own + 1]
                    spread[q0 + i, g] = p @ v[lo:own + 1].abs()
                    lse[q0 + i, g] = torch.logsumexp(s, 0)
                    slack[q0 + i, g] = (k[lo:own + 1].abs() @ x.abs()).max() * abs(scale)
    return out, lse, spread, slack


def attention_tolerance(out, lse, spread, slack, dim):
    """Bounds on |out - exact| and |lse - exact|.

    A score is a sum of dim products held in fp32 and one scaling:
    delta = (dim + 4) 2^-24 sum|q k| scale.  Each probability is then off by a
    factor exp(delta), its own exp2 and rescales by 2^-20 in all, and is rounded
    to bf16 (half a step); the sums over up to 2^14 keys run in fp32 tiles
    (2^-14).  Numerator and denominator both carry delta.  The output is
    rounded to bf16."""
    delta = (dim + 4) * 2.0 ** -24 * slack
    rel = BF16_HALF + 2.0 * delta + 2.0 ** -13
    tol = rel[..., None] * spread * (1 + BF16_HALF) + BF16_HALF * out.abs() + 2.0 ** -126
    lse_tol = delta + 2.0 ** -13 + 2.0 ** -22 * lse.abs()
    return tol, lse_tol


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Token per row from the definition, in numpy float64."""
    logits = np.asarray(logits, dtype=np.float32)
    m, n = logits.shape
    picks = []
    for i in range(m):
        row = logits[i].astype(np.float64)
        t = 1.0 if temperature is None else float(np.float32(temperature[i]))
        if np.isnan(row).any():
            picks.append(int(np.argmax(np.isnan(row))))
            continue
        top = row.max()
        if not t > 0 or top == -np.inf:
            picks.append(int(np.argmax(row)))
            continue
        with np.errstate(invalid="ignore", over="ignore", under="ignore"):
            w = np.where(row == top, 1.0, np.where(row == -np.inf, 0.0, np.exp((row - top) / t)))
        order = np.argsort(-row, kind="stable")
        k = n if top_k is None or top_k[i] <= 0 else min(int(top_k[i]), n)
        order = order[:k]
        ws = w[order]
        p = 1.0 if top_p is None else float(np.float32(top_p[i]))
        if p < 1:
            before = np.cumsum(ws) - ws
            keep = before < p * ws.sum()
            keep[0] = True
            order, ws = order[keep], ws[keep]
        floor = 0.0 if min_p is None else min(1.0, float(np.float32(min_p[i])))
        keep = np.zeros(n, bool)
        keep[order[ws >= floor]] = True
        cum = np.cumsum(np.where(keep, w, 0.0))
        target = float(np.float32(u[i])) * cum[-1]
        past = np.nonzero(cum > target)[0]
        picks.append(int(past[0]) if len(past) else int(np.argmax(row)))
    return np.array(picks, np.int32)
