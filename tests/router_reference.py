"""The router's formulas in 64 bits, one token at a time, for the tests."""
import math

import numpy as np
import torch


def scores(l, sigmoid):
    """Scores and shares of one token's logits (float64 numpy)."""
    with np.errstate(all="ignore"):
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-l))
            total = s.sum()
            return s, s / total if total else np.zeros_like(s)
        m = l[~np.isnan(l)].max(initial=-np.inf)
        x = np.where(l == -np.inf, 0.0, np.exp(l - m))
        total = x.sum()
        s = x / total if total != 0 else np.zeros_like(x)
        return s, s


def choose(l, bias, r):
    """Indices of the experts a token chooses, highest first; fewer than k where none is left."""
    s, _ = scores(l, r.score == 1)
    lowest = -np.finfo(np.float64 if bias is not None or r.group_best == 2 else np.float32).max
    key = l.copy() if bias is None and r.group_best == 1 else s + (0.0 if bias is None else bias)
    key[np.isnan(key)] = lowest
    open_ = l != -np.inf
    if bias is not None:
        open_ &= bias != -np.inf
    size = r.num_experts // r.num_groups
    if r.num_groups > 1:
        best = []
        for g in range(r.num_groups):
            inside = sorted((key[e] for e in range(g * size, (g + 1) * size) if open_[e]), reverse=True)
            best.append(max(sum(inside[:r.group_best]), lowest) if inside else None)
        order = sorted((g for g in range(r.num_groups) if best[g] is not None), key=lambda g: (-best[g], g))
        keep = set(order[:r.topk_groups])
        open_ &= np.array([e // size in keep for e in range(r.num_experts)])
    order = sorted(np.nonzero(open_)[0], key=lambda e: (-key[e], e))
    return [int(e) for e in order[:r.num_topk]]


def route(logits, bias, mask, r):
    """(ids, weights) of all tokens; logits in any type, on any device."""
    l = logits.detach().double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    ids = np.full((l.shape[0], r.num_topk), -1, np.int64)
    w = np.zeros((l.shape[0], r.num_topk))
    for t in range(l.shape[0]):
        if mask is not None and not bool(mask[t]):
            continue
        chosen = choose(l[t], b, r)
        s, _ = scores(l[t], r.score == 1)
        part = s[chosen]
        if r.renormalize:
            part = part / (part.sum() + 1e-20)
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = r.scale * part
    return ids, w


def ranges(T, off):
    if off is None:
        return [(0, T)]
    off = [int(o) for o in off]
    return [(max(0, a), min(T, b)) for a, b in zip(off, off[1:])]


def balance(logits, idx, off, r):
    """(loss, counts, coef), and the share sums, in 64 bits."""
    l, ids = logits.detach().double().cpu().numpy(), idx.cpu().numpy()
    parts, E = ranges(l.shape[0], off), r.num_experts
    counts, sums, tokens = np.zeros((len(parts), E), np.int64), np.zeros((len(parts), E)), np.zeros(len(parts))
    for q, (a, b) in enumerate(parts):
        for t in range(a, b):
            live = [int(i) for i in ids[t] if 0 <= i < E]
            if live:
                np.add.at(counts[q], live, 1)
                sums[q] += scores(l[t], r.score == 1)[1]
                tokens[q] += 1
    used = max(1, int((tokens > 0).sum()))
    coef = np.array([E / (r.num_topk * n * n * used) if n else 0.0 for n in tokens])
    return float((coef * (counts * sums).sum(1)).sum()), counts, coef, sums


def backward(logits, idx, grad_w, counts, coef, grad_loss, off, r):
    """(gradient, magnitude of the terms it is the sum of), in 64 bits."""
    l, ids = logits.detach().double().cpu().numpy(), idx.cpu().numpy()
    T, E = l.shape
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    at = np.full(T, -1)
    for q, (a, b) in enumerate(ranges(T, off)):
        at[a:max(a, b)] = q
    for t in range(T):
        live = [(j, int(i)) for j, i in enumerate(ids[t]) if 0 <= i < E]
        if not live:
            continue
        s, p = scores(l[t], r.score == 1)
        n, g, ga = np.zeros(E), np.zeros(E), np.zeros(E)
        if grad_w is not None:
            for j, i in live:
                n[i] += 1
                g[i] += float(grad_w[t, j])
                ga[i] += abs(float(grad_w[t, j]))
        if r.renormalize and n.any():
            D = (n * s).sum() + 1e-20
            u = r.scale * (g - n * (g * s).sum() / D) / D
            ua = abs(r.scale) * (ga + n * (ga * s).sum() / D) / D
        else:
            u, ua = r.scale * g, abs(r.scale) * ga
        b, ba = np.zeros(E), np.zeros(E)
        if counts is not None and at[t] >= 0:
            c, f = counts[at[t]].double().cpu().numpy(), float(coef[at[t]]) * float(grad_loss)
            b, ba = f * (c - (p * c).sum()), abs(f) * (abs(c - c[0]) + (p * abs(c - c[0])).sum())
        if r.score == 1:
            total = s.sum()
            inv = 1.0 / total if total else 0.0
            slope = np.where(np.isfinite(l[t]), np.exp(-abs(l[t])) / (1.0 + np.exp(-abs(l[t]))) ** 2, 0.0)
            grad[t], size[t] = slope * (u + b * inv), slope * (ua + ba * inv)
        else:
            u, ua = u + b, ua + ba
            grad[t], size[t] = s * (u - (s * u).sum()), s * (ua + (s * ua).sum())
    return grad, size


def spread(logits):
    """Largest distance of a token's finite logits: what an exponent's argument may be off by, in units of
    2^-24. At most 400: exponentials below 2^-160 are zero on either side of any comparison."""
    l = logits.detach().double().cpu()
    l = l[torch.isfinite(l)]
    return min(400.0, float(l.max() - l.min()) + float(l.abs().max())) if l.numel() else 0.0


def close(got, want, tol, what):
    """|got - want| <= tol, elementwise; NaN and infinities have to be the same."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    with np.errstate(invalid="ignore"):
        off = np.where(fine, abs(got - want) - tol, -math.inf)
    assert off.size == 0 or off.max() <= 0, "%s: %g past the bound at %s" % (what, off.max(), np.unravel_index(off.argmax(), off.shape))
