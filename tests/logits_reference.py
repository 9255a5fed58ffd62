"""Plain 64-bit implementations of the logits operators, row by row in numpy, and the error
bounds of the 32-bit kernels against them.

The implementations follow the definitions in include/argreduce.h and share nothing with the
library. Inputs are float64 copies of the stored logits, so both sides start from the same
numbers.

Error bounds. u = 2^-24 is half a binary32 step. A kernel forms z = (x - m) * k with three
roundings (k, the difference, the product): |dz| <= 3 u |z|. A term 2^z is then off by at most
(3 u |z| ln 2 + 2 u) of itself (v_exp_f32 is good to one step, 2 u), and a sum of n terms of one
sign by another n u of itself. So log2 s is off by at most
    u (3 E|z| + n + 2) / ln 2 + 2 u log2 s      with E|z| = sum p |z|,
where the last term is v_log_f32's step and the subtraction's. A lane adds at most
cols / 64 terms (16 in a group of lanes) and the merges at most 64 more: n = cols / 64 + 80.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24
LN2 = math.log(2.0)
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# half the distance of the smallest subnormals, or binary32's flush of 2^z below 2^-126
TINY = {"f32": 2.0 ** -125, "f16": 2.0 ** -25, "bf16": 2.0 ** -125}


LOWEST = -float(np.finfo(np.float32).max)


def in_range(lp):
    """A log probability as binary32 can hold it: -inf below the lowest finite value."""
    return np.where(np.asarray(lp) < LOWEST, -np.inf, lp)


def adds(cols: int) -> float:
    return cols / 64 + 80


def softmax_row(x: np.ndarray, temperature: float):
    """(state, z, log_s, p) of a row: z = (x - max) / T; state 'ok', 'empty' or 'nan'."""
    if np.isnan(x).any() or (x == np.inf).any():
        return "nan", None, None, None
    m = x.max()
    if m == -np.inf:
        return "empty", None, None, None
    z = (x - m) / temperature
    e = np.exp(z)
    s = e.sum()
    return "ok", z, math.log(s), e / s


def logprobs_row(x, token, temperature, top):
    """dict(logprob, entropy, top [(logprob, token)], p, z, tol_*), or a special row's values."""
    none = [(-math.inf, -1)] * top
    if token < 0:
        return dict(kind="left out", logprob=0.0, entropy=0.0, top=none)
    state, z, log_s, p = softmax_row(x, temperature)
    if state == "nan":
        return dict(kind="nan", logprob=math.nan, entropy=math.nan, top=[(math.nan, -1)] * top)
    beyond = token >= len(x)
    if state == "empty":
        return dict(kind="empty", logprob=math.nan if beyond else -math.inf, entropy=0.0, top=none)
    live = p > 0
    entropy = log_s - float((p[live] * z[live]).sum())
    order = np.lexsort((np.arange(len(x)), -x))[:top]
    best = [(float(in_range(z[i] - log_s)), int(i)) for i in order if x[i] > -np.inf]
    best += [(-math.inf, -1)] * (top - len(best))
    logprob = math.nan if beyond else float(in_range(z[token] - log_s))
    ez = float((p[live] * -z[live]).sum()) / LN2  # E|z| in base 2
    n = adds(len(x))
    tol_ls = U * (3 * ez + n + 2) + 2 * U * abs(log_s)  # of ln s
    return dict(kind="ok", logprob=logprob, entropy=entropy, top=best, p=p, z=z, log_s=log_s,
                beyond=beyond, tol_ls=tol_ls,
                # h / s: h off by (n + 3 + 3 E|z|) u of itself, s by its own error
                tol_entropy=tol_ls + ez * LN2 * (tol_ls + U * (2 * n + 3 * ez + 8)) + 4 * U * abs(entropy))


def tol_logprob(row, lp):
    """Bound on a log probability lp = z - ln s of an ok row."""
    return row["tol_ls"] + 8 * U * (abs(lp) + abs(row["log_s"]))


def logprobs_grad_row(row, x, token, temperature, g, e, dtype):
    """(gradient, bound) of one row for d logprob = g, d entropy = e (None: not asked for)."""
    if row["kind"] in ("left out", "empty"):
        return np.zeros(len(x)), np.zeros(len(x))
    if row["kind"] == "nan" or row["beyond"]:
        return np.full(len(x), np.nan), np.zeros(len(x))
    p, log_s = row["p"], row["log_s"]
    z = np.maximum(row["z"], -1e5)  # masked elements: p is 0
    lp = z - log_s
    h = row["entropy"]
    d = -p * g
    size = p * abs(g)
    if e is not None:
        d = d - e * p * np.where(p > 0, lp + h, 0.0)
        size = size + abs(e) * p * (np.abs(lp) + abs(h) + 1)
    one = np.zeros(len(x))
    one[token] = g
    d = (d + one) / temperature
    rel = row["tol_ls"] + U * (3 * np.abs(z) / LN2 + 12)
    tol = size * rel / temperature + 6 * U * np.abs(one) / temperature
    if e is not None:
        tol = tol + abs(e) * p * (row["tol_entropy"] + row["tol_ls"]) / temperature
    tol = 1.01 * tol + HALF_STEP[dtype] * (np.abs(d) + tol) + \
        TINY[dtype] * (1 + (abs(g) + abs(e or 0.0) * (abs(h) + 100)) / temperature)
    return d, tol


def distill_row(x, ids, v, temperature):
    """dict(kind, loss, q by position, tol) of one row."""
    cols = len(x)
    v = np.where(ids >= 0, v, -np.inf).astype(np.float64)
    if np.isnan(v).any() or (v == np.inf).any():
        return dict(kind="nan", loss=math.nan)
    if v.max() == -np.inf:
        return dict(kind="absent", loss=0.0)
    state, z, log_s, p = softmax_row(x, temperature)
    w = (v - v.max()) / temperature
    e = np.exp(w)
    q = e / e.sum()
    lq = w - math.log(e.sum())
    beyond = bool(((ids >= cols) & (q > 0)).any())
    if state == "nan" or beyond:
        return dict(kind="nan", loss=math.nan)
    if state == "empty":
        return dict(kind="empty", loss=math.inf)
    has = q > 0
    lp = in_range(z[np.where(has, ids, 0)] - log_s)
    loss = float((q[has] * (lq[has] - lp[has])).sum())
    at = np.zeros(cols)
    np.add.at(at, ids[has], q[has])
    live = p > 0
    ez = float((p[live] * -z[live]).sum()) / LN2
    n = adds(cols)
    tol_ls = U * (3 * ez + n + 2) + 2 * U * abs(log_s)
    k = len(ids)
    eq = float((q[has] * -w[has]).sum()) / LN2
    tol_q = U * (3 * eq + k + 82) + 2 * U * abs(math.log(e.sum()))  # of the teacher's ln sum
    size = float((q[has] * (np.abs(lq[has]) + np.abs(np.where(np.isfinite(lp[has]), lp[has], 0.0)) +
                            abs(log_s))).sum())
    tol = tol_ls + tol_q * (1 + size) + U * size * (k + 3 * float(np.abs(w[has]).max()) + 24)
    return dict(kind="ok", loss=loss, at=at, p=p, z=z, tol=1.01 * tol, tol_ls=tol_ls, tol_q=tol_q)


def distill_grad_row(row, x, temperature, g, dtype):
    if row["kind"] in ("absent", "empty"):
        return np.zeros(len(x)), np.zeros(len(x))
    if row["kind"] == "nan":
        return np.full(len(x), np.nan), np.zeros(len(x))
    d = g / temperature * (row["p"] - row["at"])
    z = np.maximum(row["z"], -1e5)
    tol = abs(g) / temperature * (row["p"] * (row["tol_ls"] + U * (3 * np.abs(z) / LN2 + 12)) +
                                  row["at"] * (row["tol_q"] + 1100 * U))
    tol = 1.01 * tol + HALF_STEP[dtype] * (np.abs(d) + tol) + TINY[dtype] * (1 + abs(g) / temperature)
    return d, tol


def agree(got, want, tol, what):
    """got within tol of want; NaN and infinities exactly where want has them."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    rest = ~fine & ~np.isnan(want)
    assert np.array_equal(got[rest], want[rest]), f"{what}: infinities elsewhere"
    off = np.abs(got[fine] - want[fine])
    bad = ~(off <= tol[fine])
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off; worst {off[bad].max():.3g} where "
                           f"{tol[fine][bad][off[bad].argmax()]:.3g} is allowed")
