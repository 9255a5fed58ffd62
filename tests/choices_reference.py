"""Plain 64-bit implementations of beam search's step and reordering and of expert routing, in numpy, and
the error bounds of the 32-bit kernels against them.

They follow the definitions in include/argreduce.h and share nothing with the library.

Bounds, with u = 2^-24 and the terms of logits_reference (a sum of exponentials: an argument z is off by at most
3 u |z|, a term by 2 u more, n additions by n u): ``tol_ls`` there bounds ln s. A beam's value has the rounding of k
taken out and its logarithm in binary64, so the same bound holds for it with room; the value is rounded once, u of
itself. Probabilities are p (1 +- rel), rel = tol_ls + u (3 |z| / ln 2 + 12), as for the gradients there.
"""
from __future__ import annotations

import math

import numpy as np

import logits_reference as R

U = R.U


def beam_values(x, scores, ended, end_token, temperature):
    """[(value, beam, token, bound, row key, logit)] of one group, best first: by value, beam, logit and token. Rows
    with equal keys are the same row with the same score: their values are equal, not just close."""
    out = []
    for b, row in enumerate(x):
        s = float(scores[b])
        if not math.isfinite(s):
            continue
        if ended is not None and ended[b]:
            out.append((s, b, end_token, 0.0, ("ended", s), 0.0))
            continue
        state, z, log_s, p = R.softmax_row(row, temperature)
        if state != "ok":
            continue
        live = p > 0
        ez = float((p[live] * -z[live]).sum()) / math.log(2.0)
        tol = U * (3 * ez + R.adds(len(row)) + 2) + 1e-15 * (abs(s) + np.abs(z).max(initial=0, where=np.isfinite(z)))
        key = (s, row.tobytes())
        for v in np.flatnonzero(row > -np.inf):
            out.append((s + (float(z[v]) - log_s), b, int(v), tol, key, float(row[v])))
    out.sort(key=lambda c: (-c[0], c[1], -c[5], c[2]))
    return out


def check_beam_group(got, want, width, what):
    """got: (scores, parents, tokens) of one group. Equal to the best of `want` in order, but where values of
    different rows lie within their bounds of each other either order is right."""
    scores, parents, tokens = got
    n = min(width, len(want))
    assert [int(p) for p in parents[n:]] == [-1] * (width - n), what
    assert [int(t) for t in tokens[n:]] == [-1] * (width - n), what
    assert all(s == -math.inf for s in scores[n:]), what
    at = {(b, t): i for i, (_, b, t, *_) in enumerate(want)}
    seen = set()
    for j in range(n):
        place = (int(parents[j]), int(tokens[j]))
        assert place in at, f"{what}: {place} is not offered"
        assert place not in seen, f"{what}: {place} twice"
        seen.add(place)
        i = at[place]
        if i != j:
            a, b = want[min(i, j)], want[max(i, j)]
            assert a[4] != b[4] or a[3] == 0.0, f"{what}: candidate {j} is {place}, want {want[j][1:3]}"
            assert a[0] - b[0] <= a[3] + b[3], f"{what}: candidate {j} is {place}, want {want[j][1:3]}"
        value, tol = want[i][0], want[i][3]
        bound = tol + 2.0 ** -24 * abs(value) + 2.0 ** -149
        if value < R.LOWEST:
            assert scores[j] == -math.inf, what
        else:
            assert abs(float(scores[j]) - value) <= bound, f"{what}: score {scores[j]} for {value}"


def reorder(state, parents, dim, first, last):
    """A copy of `state` (numpy, [groups, beams, ...]) after the move; dim None: no positions."""
    out = state.copy()
    groups, beams = parents.shape
    for g in range(groups):
        n = state.shape[dim] if dim is not None else 1
        a, b = max(0, int(first[g])), min(n, int(last[g]))
        if a >= b:
            continue
        cut = (Ellipsis,) if dim is None else (slice(None),) * (dim - 2) + (slice(a, b),)
        for k in range(beams):
            p = int(parents[g, k])
            if 0 <= p < beams:
                out[(g, k) + cut] = state[(g, p) + cut]
    return out


def route_group(x, live, top, renormalize):
    """One group of tokens: dict with per-token lists and the totals, and what the bounds need."""
    tokens, experts = x.shape
    out = dict(experts=np.full((tokens, top), -1), weights=np.zeros((tokens, top)), tol_w=np.zeros((tokens, top)),
               counts=np.zeros(experts, dtype=np.int64), rows=[None] * tokens, n=0)
    share, share_tol, z, z_tol = np.zeros(experts), np.zeros(experts), 0.0, 0.0
    for t in range(tokens):
        if not live[t]:
            continue
        state, zz, log_s, p = R.softmax_row(x[t], 1.0)
        if state == "empty":
            continue
        out["n"] += 1
        if state == "nan":
            out["experts"][t], out["weights"][t] = -2, math.nan
            out["rows"][t] = "nan"
            share[:], z = math.nan, math.nan
            continue
        at = p > 0
        ez = float((p[at] * -zz[at]).sum()) / math.log(2.0)
        tol_ls = U * (3 * ez + R.adds(experts) + 2) + 2 * U * abs(log_s)
        rel = tol_ls + U * (3 * np.minimum(-zz, 1e5) / math.log(2.0) + 12)
        order = np.lexsort((np.arange(experts), -x[t]))[:top]
        order = order[x[t][order] > -np.inf]
        k = len(order)
        w, tw = p[order], p[order] * rel[order]
        if renormalize:
            kept = p[order].sum()
            tw = (w * (rel[order] + (p[order] * rel[order]).sum() / kept + 80 * U)) / kept
            w = w / kept
        out["experts"][t, :k], out["weights"][t, :k], out["tol_w"][t, :k] = order, w, 1.01 * tw + 2.0 ** -126
        out["counts"][order] += 1
        share += p
        share_tol += p * rel
        lse = float(x[t].max()) + log_s
        e = tol_ls + 4 * U * (abs(lse) + abs(log_s) + abs(float(x[t].max())))
        z += lse * lse
        z_tol += 2 * abs(lse) * e + e * e
        out["rows"][t] = dict(p=p, rel=rel, lse=lse, tol_lse=e, chosen=order)
    n = out["n"]
    adds = (tokens + 600) * U
    scale = experts / (top * n * n) if n else 0.0
    out["scale"] = scale
    out["balance"] = scale * float((out["counts"] * share).sum()) if n else 0.0
    out["tol_balance"] = 1.01 * (scale * float((out["counts"] * share_tol).sum()) + adds * abs(out["balance"]))
    out["z"] = z / n if n else 0.0
    if out["z"] > -R.LOWEST:  # past binary32
        out["z"] = math.inf
    out["tol_z"] = 1.01 * (z_tol / n + adds * abs(out["z"])) + 2.0 ** -126 if n else 0.0
    return out


def route_grad_token(group, t, renormalize, gw, g_balance, g_z, dtype):
    """(gradient, bound) of one token's logits."""
    row, experts = group["rows"][t], len(group["counts"])
    if row is None:
        return np.zeros(experts), np.zeros(experts)
    if isinstance(row, str):
        return np.full(experts, math.nan), np.zeros(experts)
    p, rel, c, order = row["p"], row["rel"], group["counts"].astype(np.float64), row["chosen"]
    gw = np.asarray(gw, dtype=np.float64)[:len(order)]
    pb, pz = group["scale"] * g_balance, 2 * g_z / group["n"]
    even, even_tol = float((c * p).sum()), float((c * p * rel).sum())
    factor = pb * (c - even) + pz * row["lse"]
    size = abs(pb) * (c + even) + abs(pz * row["lse"])
    less = abs(pb) * even_tol + abs(pz) * row["tol_lse"]
    q = p[order]
    d, tol = np.zeros(experts), np.zeros(experts)
    if renormalize:
        kept = q.sum()
        w = q / kept
        inside, big = float((gw * w).sum()), float((np.abs(gw) * w).sum())
        rel_w = rel[order] + float((q * rel[order]).sum()) / kept + 100 * U
        np.add.at(d, order, w * (gw - inside))
        np.add.at(tol, order, w * ((np.abs(gw) + big) * 2 * rel_w + float((np.abs(gw) * w * rel_w).sum())))
    else:
        inside, big = float((gw * q).sum()), float((np.abs(gw) * q).sum())
        factor, size = factor - inside, size + big
        less += float((np.abs(gw) * q * rel[order]).sum())
        np.add.at(d, order, q * gw)
        np.add.at(tol, order, q * np.abs(gw) * (rel[order] + 12 * U))
    d = d + p * factor
    tol = tol + p * (rel * size + less + (100 + experts / 64) * U * size)
    tol = 1.01 * tol + 4 * U * np.abs(d)
    most = {"f32": -R.LOWEST, "f16": 65519.0, "bf16": 3.3961e38}[dtype]  # what still rounds to a finite value
    assert not (np.abs(np.abs(d) - most) <= tol).any()
    tol = np.where(np.abs(d) > most, 0.0, tol)
    d = np.where(np.abs(d) > most, np.copysign(np.inf, d), d)
    size = np.minimum(size, -R.LOWEST)
    tol = tol + R.HALF_STEP[dtype] * (np.where(np.isfinite(d), np.abs(d), 0.0) + tol) + \
        R.TINY[dtype] * (1 + size + np.abs(gw).max(initial=0.0))
    return d, tol
