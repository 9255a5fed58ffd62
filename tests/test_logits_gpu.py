"""The logits operators on the GPU against the plain 64-bit reference (logits_reference.py), whose
error bounds are derived there; special rows, ties, layouts, streams, graphs, autograd and a run of
the operators together."""
import math

import numpy as np
import pytest
import torch

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B
import logits_reference as R
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf


@pytest.fixture
def capacity():
    yield B.argreduce_debug_set_capacity
    B.argreduce_debug_set_capacity(0)


def host(t):
    return t.detach().double().cpu().numpy()


def make_rows(rng, rows, cols, dtype, std=2.0):
    """Ordinary rows, and among them: masked, empty, constant, the lowest value throughout, one
    that the lowest value masks, NaN, +inf, ascending, a few values only."""
    x = rng.normal(size=(rows, cols)) * std
    low = torch.finfo(DT[dtype]).min
    for r in range(rows):
        kind = r % 11
        if kind == 1:
            x[r, rng.random(cols) < 0.4] = -INF
        elif kind == 2 and rows > 3:
            x[r] = -INF
        elif kind == 3:
            x[r] = 0.25
        elif kind == 4:
            x[r] = low
        elif kind == 5:
            x[r, rng.random(cols) < 0.5] = low
        elif kind == 6 and rows > 8:
            x[r, int(rng.integers(cols))] = math.nan
        elif kind == 7 and rows > 8:
            x[r, int(rng.integers(cols))] = INF
        elif kind == 8:
            x[r] = np.arange(cols) % 97
        elif kind == 9:
            x[r] = rng.integers(0, 3, size=cols)
        elif kind == 10:
            x[r] = -INF
            x[r, int(rng.integers(cols))] = -3.0
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def check_logprobs(x, tokens, dtype, temperature=1.0, entropy=True, top=0, **kw):
    r = ar.token_logprobs(x, tokens, temperature=temperature, entropy=entropy, top=top, **kw)
    torch.cuda.synchronize()
    xs, ts = host(x).reshape(-1, x.shape[-1]), tokens.cpu().numpy().reshape(-1)
    lps, ents = host(r.logprob).reshape(-1), host(r.entropy).reshape(-1) if entropy else None
    rows = []
    for i in range(len(xs)):
        want = R.logprobs_row(xs[i], int(ts[i]), temperature, top)
        what = f"row {i} ({want['kind']})"
        ok = want["kind"] == "ok"
        R.agree(lps[i], want["logprob"], R.tol_logprob(want, want["logprob"]) if ok else 0, what)
        if entropy:
            R.agree(ents[i], want["entropy"], want["tol_entropy"] if ok else 0, what + " entropy")
        if top:
            got_t = r.top_tokens.reshape(-1, top)[i].cpu().numpy()
            got_l = host(r.top_logprobs).reshape(-1, top)[i]
            assert got_t.tolist() == [t for _, t in want["top"]], what
            wl = np.array([v for v, _ in want["top"]])
            tol = R.tol_logprob(want, np.where(np.isfinite(wl), wl, 0)) if ok else 0
            R.agree(got_l, wl, tol, what + " alternatives")
        rows.append(want)
    return r, xs, ts, rows


def check_logprobs_grad(x, tokens, dtype, temperature, entropy, r, xs, ts, rows, rng):
    lead = x.shape[:-1]
    g = torch.from_numpy(rng.normal(size=lead)).float().cuda()
    e = torch.from_numpy(rng.normal(size=lead)).float().cuda() if entropy else None
    grad = ar.token_logprobs_grad(x, tokens, r.stats, g, e, temperature=temperature)
    torch.cuda.synchronize()
    assert grad.dtype == x.dtype and grad.shape == x.shape and grad.is_contiguous()
    got, gs = host(grad).reshape(xs.shape), host(g).reshape(-1)
    es = host(e).reshape(-1) if entropy else [None] * len(xs)
    for i in range(len(xs)):
        d, tol = R.logprobs_grad_row(rows[i], xs[i], int(ts[i]), temperature, gs[i], es[i], dtype)
        R.agree(got[i], d, tol, f"gradient of row {i} ({rows[i]['kind']})")


def make_tokens(rng, rows, cols):
    t = rng.integers(0, cols, size=rows)
    if rows > 3:
        t[rows // 2] = -100
    if rows > 12:
        t[11] = cols       # the first id beyond the row
        t[0] = cols - 1
        t[12] = 2 ** 40    # far beyond
    return torch.from_numpy(t).cuda()


# Widths round the borders between lane groups, wavefronts, workgroups and splits, odd ones among
# them; with fewer columns than alternatives too.
SHAPES = [(1, 1), (4, 2), (13, 3), (13, 8), (14, 31), (23, 64), (13, 65), (13, 127), (13, 129),
          (13, 256), (14, 257), (13, 511), (13, 1000), (13, 1025), (13, 2047), (13, 2049), (12, 4100),
          (11, 8200), (11, 16411)]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_logprobs_and_gradient(dtype, rows, cols):
    rng = np.random.default_rng(rows * 1000 + cols)
    temperature = [1.0, 0.7, 3.0][cols % 3]
    top = min(64, [0, 1, 5, 20, 64][(rows + cols) % 5])
    entropy = (rows + cols) % 4 != 0
    announce(f"logprobs {dtype} [{rows},{cols}] T={temperature} top={top} entropy={entropy}")
    x = make_rows(rng, rows, cols, dtype)
    tokens = make_tokens(rng, rows, cols)
    got = check_logprobs(x, tokens, dtype, temperature, entropy, top)
    check_logprobs_grad(x, tokens, dtype, temperature, entropy, *got, rng)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("cap", [2048, 256 * 2048])
@pytest.mark.parametrize("rows,cols", [(11, 6000), (11, 20001), (3, 70001), (2, 262144)])
def test_every_path(capacity, dtype, cap, rows, cols):
    """A small simulated device takes a workgroup per row where the real one splits the row."""
    rng = np.random.default_rng(cols)
    assert capacity(cap) == 0
    plan = B.argreduce_logprobs_plan(rows, cols, dtype)
    announce(f"logprobs {dtype} [{rows},{cols}] capacity {cap}: path {plan['path']} "
             f"lanes {plan['lanes_per_row']}")
    x = make_rows(rng, rows, cols, dtype)
    tokens = make_tokens(rng, rows, cols)
    for top in (0, 7, 64):
        got = check_logprobs(x, tokens, dtype, 1.0, top != 0, top)
    check_logprobs_grad(x, tokens, dtype, 1.0, True, *got, rng)


@pytest.mark.parametrize("cap", [2048, 256 * 2048])
@pytest.mark.parametrize("cols", [40, 500, 1500, 30000, 140000])
def test_alternatives_of_tied_rows(capacity, cap, cols):
    """Rows whose ties put far more elements at the threshold than any buffer holds."""
    capacity(cap)
    announce(f"ties cols={cols} capacity {cap}")
    rng = np.random.default_rng(7)
    x = np.zeros((8, cols))
    x[1] = np.arange(cols)            # ascending: every element beats those before it
    x[2] = -np.arange(cols)
    x[3] = np.arange(cols) // 64
    x[4] = rng.integers(0, 2, size=cols)
    x[5, cols // 2:] = -INF
    x[6] = (np.arange(cols) % 256) // 32
    x[7, 0::2] = -0.0                 # equal to +0
    for dtype in sorted(DT):
        t = torch.from_numpy(x).to(DT[dtype]).cuda()
        check_logprobs(t, torch.zeros(8, dtype=torch.int64).cuda(), dtype, 1.0, True, 64)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("offset", [1, 3, 5])
@pytest.mark.parametrize("cols,pad", [(50, 14), (64, 0), (1000, 1), (3001, 7), (9001, 8)])
def test_strides_and_alignment(dtype, offset, cols, pad):
    """Rows further apart than their length, starting at any element's address."""
    rows = 13
    rng = np.random.default_rng(offset * cols)
    announce(f"strides {dtype} cols={cols} pad={pad} offset={offset}")
    buf = torch.full((rows * (cols + pad) + offset + 16,), 1e4, dtype=DT[dtype], device="cuda")
    x = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    x.copy_(make_rows(rng, rows, cols, dtype))
    tokens = make_tokens(rng, rows, cols)
    got = check_logprobs(x, tokens, dtype, 1.0, True, 5)
    check_logprobs_grad(x, tokens, dtype, 1.0, True, *got, rng)
    ids, v = make_teacher(rng, rows, cols, 9)
    check_distill(x, ids, v, dtype, 1.0, rng)
    # a gradient buffer at any element's address
    out = torch.full((rows * cols + offset + 8,), 7.0, dtype=DT[dtype], device="cuda")
    view = out[offset:offset + rows * cols].view(rows, cols)
    g = torch.ones(rows, device="cuda")
    want = ar.token_logprobs_grad(x, tokens, got[0].stats, g)
    ar.token_logprobs_grad(x, tokens, got[0].stats, g, out=view)
    assert torch.equal(view.nan_to_num(9.0), want.nan_to_num(9.0))
    assert (out[:offset] == 7).all() and (out[offset + rows * cols:] == 7).all()
    loss, want = ar.distill_step(x, ids, v, g)
    out.fill_(7.0)
    ar.distill_step(x, ids, v, g, out=view)
    assert torch.equal(view.nan_to_num(9.0), want.nan_to_num(9.0))
    assert (out[:offset] == 7).all() and (out[offset + rows * cols:] == 7).all()


def make_teacher(rng, rows, cols, k):
    ids = rng.integers(0, cols, size=(rows, k))  # equal ids among them
    v = rng.normal(size=(rows, k)) * 3
    ids[rng.random((rows, k)) < 0.1] = -1
    v[rng.random((rows, k)) < 0.05] = -INF
    if rows > 2:
        ids[1] = -1                   # no entry
        v[2] = -INF                   # no weight
    if rows > 10:
        ids[8, 0], v[8, 0] = cols, 1.0
        ids[9, 0], v[9, 0] = 0, math.nan
        ids[10] = int(rng.integers(cols))  # one id only
        v[10] = 1.0
        ids[3, 0], v[3, 0] = -1, math.nan  # an absent entry's value does not matter
    return torch.from_numpy(ids).cuda(), torch.from_numpy(v).float().cuda()


def check_distill(x, ids, v, dtype, temperature, rng):
    lead, cols = x.shape[:-1], x.shape[-1]
    w = torch.from_numpy(rng.normal(size=lead)).float().cuda()
    got = ar.distill_loss(x, ids, v, temperature=temperature)
    grad = ar.distill_loss_grad(x, ids, v, got.stats, w, temperature=temperature)
    loss, step_grad = ar.distill_step(x, ids, v, w, temperature=temperature)
    torch.cuda.synchronize()
    k = ids.shape[-1]
    xs, ws = host(x).reshape(-1, cols), host(w).reshape(-1)
    i_s, vs = ids.cpu().numpy().reshape(-1, k), host(v).reshape(-1, k)
    for i in range(len(xs)):
        want = R.distill_row(xs[i], i_s[i], vs[i], temperature)
        what = f"row {i} ({want['kind']})"
        tol = want.get("tol", 0)
        R.agree(host(got.loss).reshape(-1)[i], want["loss"], tol, what)
        R.agree(host(loss).reshape(-1)[i], want["loss"], tol, what + " step")
        d, tol = R.distill_grad_row(want, xs[i], temperature, ws[i], dtype)
        R.agree(host(grad).reshape(-1, cols)[i], d, tol, what + " gradient")
        R.agree(host(step_grad).reshape(-1, cols)[i], d, tol, what + " step's gradient")


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rows,cols,k", [(1, 1, 1), (3, 2, 3), (12, 7, 5), (13, 64, 64), (13, 65, 1),
                                         (13, 500, 33), (12, 1030, 300), (12, 2050, 1024), (11, 4099, 8),
                                         (11, 9000, 257), (3, 40001, 64)])
def test_distill(dtype, rows, cols, k):
    rng = np.random.default_rng(rows * 100 + cols + k)
    temperature = [1.0, 2.0, 0.8][cols % 3]
    announce(f"distill {dtype} [{rows},{cols}] k={k} T={temperature}")
    x = make_rows(rng, rows, cols, dtype)
    ids, v = make_teacher(rng, rows, cols, k)
    check_distill(x, ids, v, dtype, temperature, rng)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("cap", [2048, 256 * 2048])
def test_distill_every_path(capacity, dtype, cap):
    capacity(cap)
    rng = np.random.default_rng(5)
    for rows, cols in [(11, 6000), (3, 70001)]:
        announce(f"distill {dtype} [{rows},{cols}] capacity {cap}: "
                 f"path {B.argreduce_distill_plan(rows, cols, dtype)['path']}")
        x = make_rows(rng, rows, cols, dtype)
        ids, v = make_teacher(rng, rows, cols, 40)
        check_distill(x, ids, v, dtype, 1.5, rng)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rows,cols,k", [(23, 300, 7), (23, 90, 100), (13, 90, 1024), (23, 3000, 64),
                                         (13, 3000, 65), (9, 9001, 200), (9, 33000, 33), (7, 33000, 300),
                                         (5, 70001, 64)])
def test_distill_teams_go_through_several_rows(capacity, dtype, rows, cols, k):
    """One CU's worth of workgroups: each takes several rows of every kind, one after another."""
    capacity(2048)
    announce(f"distill {dtype} [{rows},{cols}] k={k} on one CU")
    rng = np.random.default_rng(rows * cols + k)
    x = make_rows(rng, rows, cols, dtype)
    ids, v = make_teacher(rng, rows, cols, k)
    ids[3:6] = -1  # three rows without a teacher in a row
    check_distill(x, ids, v, dtype, 1.0, rng)


@pytest.mark.parametrize("dtype,rows,cols", [("f32", 600, 30011), ("f16", 700, 50021), ("bf16", 9000, 4096),
                                             ("bf16", 70000, 520)])
def test_logits_too_large_for_the_cache(dtype, rows, cols):
    """Logits over 64 MiB, which are read past the caches, and more rows than are in flight at once;
    every row against 64-bit torch, a sample of rows against the reference and its bounds."""
    announce(f"large {dtype} [{rows},{cols}]")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn(rows, cols, device="cuda", generator=g) * 2).to(DT[dtype])
    tokens = torch.randint(0, cols, (rows,), device="cuda", generator=g)
    tokens[::17] = -1
    ids = torch.randint(0, cols, (rows, 12), device="cuda", generator=g)
    ids[::13] = -1
    v = torch.randn(rows, 12, device="cuda", generator=g) * 2
    w, e = torch.rand(rows, device="cuda", generator=g), torch.rand(rows, device="cuda", generator=g)
    r = ar.token_logprobs(x, tokens, entropy=True, top=3)
    grad = ar.token_logprobs_grad(x, tokens, r.stats, w, e)
    loss, dgrad = ar.distill_step(x, ids, v, w)
    d = ar.distill_loss(x, ids, v)
    dgrad2 = ar.distill_loss_grad(x, ids, v, d.stats, w)
    torch.cuda.synchronize()
    live = tokens >= 0
    for a in range(0, rows, 1000):
        cut = slice(a, a + 1000)
        lp = torch.log_softmax(x[cut].double(), 1)
        want = torch.where(live[cut], lp.gather(1, tokens[cut].clamp(min=0)[:, None])[:, 0], 0.0)
        # randn * 2: E|z| < 30 and |ln p| < 40; the bounds are logits_reference's
        assert (r.logprob[cut].double() - want).abs().max() < R.U * (3 * 30 + R.adds(cols) + 2 + 8 * 60)
        best, at = x[cut].float().sort(dim=1, descending=True, stable=True)
        assert torch.equal(r.top_tokens[cut], torch.where(live[cut, None], at[:, :3], -1))
        q = torch.where(ids[cut] >= 0, torch.softmax(v[cut].double(), 1), 0.0)
        want = (q * (torch.log_softmax(v[cut].double(), 1) - lp.gather(1, ids[cut].clamp(min=0)))).sum(1)
        assert (loss[cut].double() - want).abs().max() < R.U * (3 * 30 + R.adds(cols) + 8 * 100)
        assert torch.equal(loss[cut] == 0, (ids[cut] < 0).all(1))
    xs, ts, i_s = host(x[::97]), tokens[::97].cpu().numpy(), ids[::97].cpu().numpy()
    vs, ws, es = host(v[::97]), host(w[::97]), host(e[::97])
    got = [host(t[::97]) for t in (grad, dgrad, dgrad2)]
    for n in range(len(xs)):
        row = R.logprobs_row(xs[n], int(ts[n]), 1.0, 0)
        R.agree(got[0][n], *R.logprobs_grad_row(row, xs[n], int(ts[n]), 1.0, ws[n], es[n], dtype), f"row {n}")
        row = R.distill_row(xs[n], i_s[n], vs[n], 1.0)
        for t in got[1:]:
            R.agree(t[n], *R.distill_grad_row(row, xs[n], 1.0, ws[n], dtype), f"distill row {n}")


def test_offsets_beyond_32_bits():
    """Rows 2^31 + 8 elements apart: the last starts past 2^32 elements."""
    stride, cols = 2 ** 31 + 8, 1000
    announce("offsets beyond 32 bits")
    buf = torch.empty(2 * stride + cols, dtype=torch.float16, device="cuda")
    x = buf.as_strided((3, cols), (stride, 1))
    rng = np.random.default_rng(3)
    x.copy_(torch.from_numpy(rng.normal(size=(3, cols))).half().cuda())
    tokens = torch.tensor([5, 999, 0], device="cuda")
    got = check_logprobs(x, tokens, "f16", 1.0, True, 5)
    check_logprobs_grad(x, tokens, "f16", 1.0, True, *got, rng)
    check_distill(x, *make_teacher(rng, 3, cols, 7), "f16", 1.0, rng)


@pytest.mark.parametrize("rows,cols", [(1, 3_000_001), (2, 1_000_003)])
def test_very_wide_rows(rows, cols):
    announce(f"wide [{rows},{cols}]")
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(size=(rows, cols)) * 3).float().cuda()
    tokens = torch.tensor([cols - 1, 17][:rows], device="cuda")
    got = check_logprobs(x, tokens, "f32", 1.0, True, 64)
    check_logprobs_grad(x, tokens, "f32", 1.0, True, *got, rng)
    check_distill(x, *make_teacher(rng, rows, cols, 64), "f32", 1.0, rng)


def test_many_rows():
    """More rows than a device wave, short ones."""
    announce("many rows")
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.normal(size=(70000, 24)) * 2).half().cuda()
    tokens = torch.from_numpy(rng.integers(-1, 24, size=70000)).cuda()
    r = ar.token_logprobs(x, tokens, entropy=True, top=3)
    y = torch.log_softmax(x.double(), 1)
    live = tokens >= 0
    want = torch.where(live, y.gather(1, tokens.clamp(min=0)[:, None])[:, 0], 0.0)
    # rows of 24: E|z| below 30 and 81 additions (see logits_reference), log probabilities below 20
    assert (r.logprob.double() - want).abs().max() < R.U * (3 * 30 + 83 + 8 * 24)
    v, i = x.float().sort(dim=1, descending=True, stable=True)
    assert torch.equal(r.top_tokens, torch.where(live[:, None], i[:, :3], -1))


@pytest.mark.parametrize("value", [1e4, -1e4, 6e4])
def test_large_common_offset(value):
    """A constant added to a row changes nothing but the rounding of the stored logits."""
    announce(f"offset {value}")
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.normal(size=(11, 3000)) * 2 + value).float().cuda()
    tokens = make_tokens(rng, 11, 3000)
    got = check_logprobs(x, tokens, "f32", 1.0, True, 20)
    check_logprobs_grad(x, tokens, "f32", 1.0, True, *got, rng)


@pytest.mark.parametrize("temperature", [2.0 ** -60, 1e-3, 1e3, 2.0 ** 60])
def test_extreme_temperatures(temperature):
    announce(f"temperature {temperature}")
    rng = np.random.default_rng(6)
    for cols in (40, 700, 9000):
        x = torch.from_numpy(np.round(rng.normal(size=(5, cols)) * 4) / 4).float().cuda()
        tokens = torch.from_numpy(rng.integers(0, cols, size=5)).cuda()
        r = ar.token_logprobs(x, tokens, temperature=temperature, entropy=True)
        torch.cuda.synchronize()
        xs = host(x)
        for i in range(5):
            want = R.logprobs_row(xs[i], int(tokens[i]), temperature, 0)
            lp = want["logprob"]
            # beyond the range of a float the log probability is -inf
            if lp < -3e38:
                assert r.logprob[i] == -INF
            else:
                R.agree(host(r.logprob[i]), lp, R.tol_logprob(want, lp) + 3 * R.U * abs(lp), f"row {i}")
            R.agree(host(r.entropy[i]), want["entropy"], want["tol_entropy"], f"row {i} entropy")


def test_leading_dimensions_and_slices():
    announce("leading dimensions")
    rng = np.random.default_rng(8)
    full = torch.from_numpy(rng.normal(size=(3, 5, 640))).float().cuda()
    x = full[:, :, :600]
    tokens = torch.from_numpy(rng.integers(0, 600, size=(3, 5))).cuda()
    got = check_logprobs(x, tokens, "f32", 1.0, True, 4)
    assert got[0].logprob.shape == (3, 5) and got[0].top_tokens.shape == (3, 5, 4)
    check_logprobs_grad(x, tokens, "f32", 1.0, True, *got, rng)
    last = full[:, -1]  # one position of every sequence: rows 5 * 640 apart
    check_logprobs(last, tokens[:, -1].contiguous(), "f32", 1.0, True, 4)
    one = full[0, 0]
    r = ar.token_logprobs(one, tokens[0, 0], entropy=True, top=2)
    assert r.logprob.shape == () and r.top_tokens.shape == (2,)
    assert torch.equal(r.logprob, ar.token_logprobs(full[0], tokens[0], entropy=True).logprob[0]) or \
        abs(float(r.logprob) - float(torch.log_softmax(one.double(), 0)[tokens[0, 0]])) < 1e-5
    empty = ar.token_logprobs(full[:0, 0], tokens[:0, 0].contiguous(), entropy=True, top=2)
    assert empty.logprob.shape == (0,) and empty.top_tokens.shape == (0, 2)
    loss, grad = ar.distill_step(full[:0, 0], torch.zeros(0, 3, dtype=torch.int64, device="cuda"),
                                 torch.zeros(0, 3, device="cuda"), torch.zeros(0, device="cuda"))
    assert loss.shape == (0,) and grad.shape == (0, 640)


def test_refusals():
    announce("refusals")
    x = torch.zeros(4, 8, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    ids, v = torch.zeros(4, 3, dtype=torch.int64, device="cuda"), torch.zeros(4, 3, device="cuda")
    w = torch.zeros(4, device="cuda")
    bad = [lambda: ar.token_logprobs(x.double(), t), lambda: ar.token_logprobs(x.t(), t),
           lambda: ar.token_logprobs(x, t.int()), lambda: ar.token_logprobs(x, t[:3]),
           lambda: ar.token_logprobs(x, t.cpu()), lambda: ar.token_logprobs(x, t, temperature=0.0),
           lambda: ar.token_logprobs(x, t, temperature=math.nan),
           lambda: ar.token_logprobs(x, t, top=65), lambda: ar.token_logprobs(x, t, top=-1),
           lambda: ar.token_logprobs(x[:, :0], t), lambda: ar.token_logprobs(x[0, 0], t[0]),
           lambda: ar.token_logprobs(x[:1].expand(4, 8), t),
           lambda: ar.token_logprobs(x.view(2, 2, 8).transpose(0, 1), t.view(2, 2)),
           lambda: ar.token_logprobs(x, torch.zeros(8, dtype=torch.int64, device="cuda")[::2]),
           lambda: ar.token_logprobs(x, t, scratch=torch.empty(64)),
           lambda: ar.token_logprobs_grad(x, t, torch.zeros(5, 4, device="cuda"), w),
           lambda: ar.token_logprobs_grad(x, t, torch.zeros(4, 4, device="cuda"), w.double()),
           lambda: ar.token_logprobs_grad(x, t, torch.zeros(4, 4, device="cuda"), w, w[:2]),
           lambda: ar.token_logprobs_grad(x, t, torch.zeros(4, 4, device="cuda"), w, out=x.half()),
           lambda: ar.token_logprobs_grad(x, t, torch.zeros(4, 4, device="cuda"), w, out=x.view(8, 4)),
           lambda: ar.distill_loss(x, ids, v.double()), lambda: ar.distill_loss(x, ids[:, :2], v),
           lambda: ar.distill_loss(x, ids[:, :0], v[:, :0]), lambda: ar.distill_loss(x, ids.int(), v),
           lambda: ar.distill_loss(x, torch.zeros(4, 1025, dtype=torch.int64, device="cuda"),
                                   torch.zeros(4, 1025, device="cuda")),
           lambda: ar.distill_loss_grad(x, ids, v, torch.zeros(4, 4, device="cuda"), w),
           lambda: ar.distill_step(x, ids, v, w[:2]),
           lambda: ar.distill_step(x, ids, v, w, out=torch.zeros(4, 16, device="cuda")[:, ::2])]
    for n, f in enumerate(bad):
        with pytest.raises((ValueError, ar.ArgreduceError)):
            f()
            pytest.fail(f"call {n} was not refused")


def raw_logprobs(x, tokens, top, stats, lp, tok, scratch, soff, sbytes):
    return B.argreduce_logprobs(x.data_ptr(), B.F32, x.shape[0], x.shape[1], x.stride(0), tokens.data_ptr(),
                                1.0, 1, top, stats.data_ptr(), lp.data_ptr(), tok.data_ptr(),
                                scratch.data_ptr() + soff, sbytes, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("soff", [0, 1, 13])
def test_scratch_and_output_bounds(soff):
    """Nothing outside the outputs and the scratch's stated size is written; the scratch may start
    anywhere and hold anything."""
    announce(f"bounds, scratch offset {soff}")
    rows, cols, top = 3, 202048, 20
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.normal(size=(rows, cols))).float().cuda()
    tokens = torch.tensor([0, -1, cols - 1], device="cuda")
    need = B.argreduce_logprobs_scratch_bytes(rows, cols, B.F32)
    assert need > 0
    want = ar.token_logprobs(x, tokens, entropy=True, top=top)
    for fill in (0, 255, 0x7f):
        scratch = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        stats = torch.full((4 * rows + 8,), 5.0, device="cuda")
        lp = torch.full((rows * top + 8,), 5.0, device="cuda")
        tok = torch.full((rows * top + 8,), 5, dtype=torch.int64, device="cuda")
        assert raw_logprobs(x, tokens, top, stats, lp, tok, scratch, soff, need) == 0
        torch.cuda.synchronize()
        assert torch.equal(stats[:4 * rows], want.stats.reshape(-1)) and (stats[4 * rows:] == 5).all()
        assert torch.equal(lp[:rows * top], want.top_logprobs.reshape(-1)) and (lp[rows * top:] == 5).all()
        assert torch.equal(tok[:rows * top], want.top_tokens.reshape(-1)) and (tok[rows * top:] == 5).all()
        assert (scratch[:soff] == fill).all() and (scratch[soff + need:] == fill).all()


SAME = [(3, 50), (40, 900), (5, 5000), (2, 202048), (700, 40000)]


@pytest.mark.parametrize("rows,cols", SAME)
def test_same_bits_every_time(rows, cols):
    announce(f"same bits [{rows},{cols}]")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    tokens = torch.randint(0, cols, (rows,), device="cuda", generator=g)
    ids = torch.randint(0, cols, (rows, 40), device="cuda", generator=g)
    v, w = torch.randn(rows, 40, device="cuda", generator=g), torch.rand(rows, device="cuda", generator=g)

    def once():
        r = ar.token_logprobs(x, tokens, entropy=True, top=9)
        return [r.stats, r.top_logprobs, r.top_tokens, ar.token_logprobs_grad(x, tokens, r.stats, w, w),
                *ar.distill_step(x, ids, v, w)]

    first = once()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


def test_streams():
    """Calls side by side on two streams, each with scratch of its own, on tensors made on another."""
    announce("streams")
    g = torch.Generator(device="cuda").manual_seed(2)
    xs = [torch.randn(4, 202048, device="cuda", generator=g) for _ in range(2)]
    tokens = torch.randint(0, 202048, (4,), device="cuda", generator=g)
    want = [ar.token_logprobs(x, tokens, entropy=True, top=20) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(ar.token_logprobs(xs[n], tokens, entropy=True, top=20))
    torch.cuda.synchronize()
    for n in range(2):
        for r in got[n]:
            assert torch.equal(r.stats, want[n].stats) and torch.equal(r.top_tokens, want[n].top_tokens)


@pytest.mark.parametrize("rows,cols", [(6, 100), (3, 202048), (600, 20000)])
def test_graph_replay(rows, cols):
    """A captured run replayed on new inputs, with eager work between the replays."""
    announce(f"graph [{rows},{cols}]")
    x = torch.randn(rows, cols, device="cuda").half()
    tokens = torch.randint(0, cols, (rows,), device="cuda")
    ids, v = torch.randint(0, cols, (rows, 12), device="cuda"), torch.randn(rows, 12, device="cuda")
    w = torch.rand(rows, device="cuda")

    def work():
        r = ar.token_logprobs(x, tokens, entropy=True, top=6)
        g = ar.token_logprobs_grad(x, tokens, r.stats, w, w)
        return [r.stats, r.top_logprobs, r.top_tokens, g, *ar.distill_step(x, ids, v, w)]

    work()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs alive at once
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = work()
        graphs.append((graph, outs))
    for n in range(4):
        x.copy_(torch.randn(rows, cols, device="cuda").half())
        tokens.copy_(torch.randint(-1, cols, (rows,), device="cuda"))
        graph, outs = graphs[n % 2]
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = work()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {n}"


def test_autograd():
    announce("autograd")
    rng = np.random.default_rng(11)
    for dtype in sorted(DT):
        x = torch.from_numpy(rng.normal(size=(3, 4, 700))).to(DT[dtype]).cuda().requires_grad_()
        tokens = torch.from_numpy(rng.integers(0, 700, size=(3, 4))).cuda()
        g, e = torch.randn(3, 4, device="cuda"), torch.randn(3, 4, device="cuda")
        r = ar.token_logprobs(x, tokens, temperature=0.9, entropy=True, top=3)
        assert r.logprob.requires_grad and r.entropy.requires_grad
        assert not r.top_logprobs.requires_grad and not r.stats.requires_grad
        (r.logprob * g + r.entropy * e).sum().backward()
        want = ar.token_logprobs_grad(x.detach(), tokens, r.stats, g, e, temperature=0.9)
        assert torch.equal(x.grad, want)
        for pick in ("logprob", "entropy"):  # one output alone
            x.grad = None
            r = ar.token_logprobs(x, tokens, entropy=True)
            (getattr(r, pick) * g).sum().backward()
            z = torch.zeros_like(g)
            want = ar.token_logprobs_grad(x.detach(), tokens, r.stats, *((g, z) if pick == "logprob" else (z, g)))
            assert torch.allclose(x.grad, want, rtol=2 * R.HALF_STEP[dtype], atol=1e-6)
        ids, v = torch.randint(0, 700, (3, 4, 5), device="cuda"), torch.randn(3, 4, 5, device="cuda")
        x.grad = None
        d = ar.distill_loss(x, ids, v, temperature=1.5)
        d.loss.backward(g)
        _, want = ar.distill_step(x.detach(), ids, v, g, temperature=1.5)
        assert torch.equal(x.grad, want)
        # an expanded gradient, and through a view of padded logits
        big = torch.zeros(6, 704, dtype=DT[dtype], device="cuda", requires_grad=True)
        ar.token_logprobs(big[:, :700], torch.zeros(6, dtype=torch.int64, device="cuda")).logprob.sum().backward()
        assert (big.grad[:, 700:] == 0).all() and (big.grad[:, 0] > 0).all() and (big.grad[:, 1:700] < 0).all()
        with torch.no_grad():
            assert not ar.token_logprobs(x, tokens).logprob.requires_grad


def test_gradient_is_the_difference():
    """The kernels' gradients against central differences of the 64-bit values."""
    announce("differences")
    rng = np.random.default_rng(12)
    cols, step = 37, 1e-4
    x = torch.from_numpy(rng.normal(size=(1, cols))).float().cuda()
    tokens = torch.tensor([5], device="cuda")
    ids, v = torch.tensor([[3, 9, 3, -1]], device="cuda"), torch.tensor([[1.0, 0.5, -1.0, 9.0]], device="cuda")
    one = torch.ones(1, device="cuda")
    r = ar.token_logprobs(x, tokens, entropy=True)
    g = host(ar.token_logprobs_grad(x, tokens, r.stats, one, one))[0]
    dg = host(ar.distill_step(x, ids, v, one)[1])[0]
    y = host(x)[0]
    for j in range(cols):
        a, b = y.copy(), y.copy()
        a[j] += step
        b[j] -= step
        f = [R.logprobs_row(t, 5, 1.0, 0) for t in (a, b)]
        diff = (f[0]["logprob"] + f[0]["entropy"] - f[1]["logprob"] - f[1]["entropy"]) / (2 * step)
        assert abs(diff - g[j]) < 30 * step ** 2 + 1e-5  # third derivative, and 32-bit arithmetic
        d = [R.distill_row(t, host(ids)[0].astype(int), host(v)[0], 1.0)["loss"] for t in (a, b)]
        assert abs((d[0] - d[1]) / (2 * step) - dg[j]) < 30 * step ** 2 + 1e-5


def test_captured_autograd_is_refused():
    announce("captured autograd")
    x = torch.randn(4, 100, device="cuda", requires_grad=True)
    tokens = torch.zeros(4, dtype=torch.int64, device="cuda")
    ids, v = torch.zeros(4, 2, dtype=torch.int64, device="cuda"), torch.zeros(4, 2, device="cuda")
    ar.token_logprobs(x, tokens).logprob.sum().backward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            ar.token_logprobs(x, tokens)
        with pytest.raises(RuntimeError, match="captured"):
            ar.distill_loss(x, ids, v)
        with torch.no_grad():
            r = ar.token_logprobs(x, tokens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.logprob, ar.token_logprobs(x.detach(), tokens).logprob)


def test_run_together():
    """A teacher's top alternatives go straight into the student's loss; the greedy answer of the
    library is the first alternative; an eager autograd step, the single call and a captured step
    agree."""
    announce("run together")
    g = torch.Generator(device="cuda").manual_seed(13)
    rows, cols, k = 24, 32003, 16
    hidden = torch.randn(rows, 64, device="cuda", generator=g)
    teacher = hidden @ torch.randn(64, cols, device="cuda", generator=g) * 0.4
    weight = (torch.randn(64, cols, device="cuda", generator=g) * 0.1).requires_grad_()
    tokens = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    greedy = ar.argmax(teacher)
    t = ar.token_logprobs(teacher, greedy, top=k)
    assert torch.equal(t.top_tokens[:, 0], greedy) and torch.equal(t.top_logprobs[:, 0], t.logprob)
    skipped = ar.token_logprobs(teacher, tokens, top=k)  # rows left out: no teacher
    ids, v = t.top_tokens.clone(), t.top_logprobs.clone()
    ids[::4], v[::4] = skipped.top_tokens[::4], skipped.top_logprobs[::4]
    logits = hidden @ weight
    d = ar.distill_loss(logits, ids, v, temperature=2.0)
    assert (d.loss[::4] == 0).all() and (d.loss[1::4] > 0).all()
    share = torch.full((rows,), 1.0 / rows, device="cuda")
    (d.loss * share).sum().backward()
    loss, grad = ar.distill_step(logits.detach(), ids, v, share, temperature=2.0)
    assert torch.equal(loss, d.loss.detach())
    # the product of the same gradient: the same call, so the same rounding
    assert torch.equal(weight.grad, hidden.t() @ grad)
    # against 64 bits: the share, q and p of each row
    p = torch.softmax(logits.detach().double() / 2, 1)
    q = torch.zeros_like(p)
    live = ids[:, 0] >= 0
    q.scatter_add_(1, ids.clamp(min=0), torch.where(live[:, None], torch.softmax(v.double() / 2, 1), 0.0).nan_to_num(0.0))
    want = (p * live[:, None] - q) / 2 / rows
    # |logits| < 40 / 2: z is off by 3 u 60, the sums by 600 u (logits_reference), times p or q <= 1
    assert (grad.double() - want).abs().max() < R.U * 1000 / rows


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rows,cols,k", [(40, 17, 128), (70, 17, 8), (9, 150, 256), (9, 2000, 200), (12, 2000, 257),
                                         (30, 600, 300), (5, 33000, 1024), (5, 33000, 17), (3, 150001, 1000)])
def test_distill_with_many_equal_ids(dtype, rows, cols, k):
    """Ids from a small part of the row, every one of them there several times, some absent."""
    announce(f"equal ids {dtype} [{rows},{cols}] k={k}")
    rng = np.random.default_rng(rows + cols + k)
    x = make_rows(rng, rows, cols, dtype)
    ids = rng.integers(0, max(1, min(cols, k) // 5), size=(rows, k)) + rng.integers(0, cols - min(cols, k) // 5 + 1)
    ids[rng.random(size=ids.shape) < 0.1] = -1
    ids = torch.from_numpy(np.minimum(ids, cols - 1)).cuda()
    ids[0] = cols - 1  # one id alone
    v = torch.from_numpy(rng.normal(size=(rows, k))).float().cuda()
    check_distill(x, ids, v, dtype, 1.0, rng)


def test_single_row_and_single_dimension():
    announce("one row")
    rng = np.random.default_rng(31)
    buf = torch.from_numpy(rng.normal(size=(1, 5000)) * 2).float().cuda()
    x = buf.as_strided((1, 5000), (2 ** 33, 1))  # the stride of a row that has no next one
    tokens = torch.tensor([17], device="cuda")
    got = check_logprobs(x, tokens, "f32", 1.0, True, 3)
    check_logprobs_grad(x, tokens, "f32", 1.0, True, *got, rng)
    ids, v = make_teacher(rng, 1, 5000, 70)
    check_distill(x, ids, v, "f32", 1.0, rng)
    loss, grad = ar.distill_step(x, ids, v, torch.ones(1, device="cuda"))
    loss1, grad1 = ar.distill_step(buf[0], ids[0], v[0], torch.ones((), device="cuda"))
    assert loss1.shape == () and grad1.shape == (5000,)
    assert loss1 == loss[0] and torch.equal(grad1, grad[0])


def test_gradient_over_the_logits_is_refused():
    announce("overlap")
    buf = torch.zeros(100, device="cuda")
    x, t = buf[:32].view(4, 8), torch.zeros(4, dtype=torch.int64, device="cuda")
    ids, v, w = t.view(4, 1), torch.zeros(4, 1, device="cuda"), torch.zeros(4, device="cuda")
    for out in (x, buf[31:63].view(4, 8)):
        with pytest.raises(ValueError, match="overlap"):
            ar.token_logprobs_grad(x, t, torch.zeros(4, 4, device="cuda"), w, out=out)
        with pytest.raises(ValueError, match="overlap"):
            ar.distill_loss_grad(x, ids, v, torch.zeros(5, 4, device="cuda"), w, out=out)
        with pytest.raises(ValueError, match="overlap"):
            ar.distill_step(x, ids, v, w, out=out)
    ar.distill_step(x, ids, v, w, out=buf[32:64].view(4, 8))


def test_backward_in_a_capture_is_refused(monkeypatch):
    """(The capture is feigned: what torch does with one whose graph was recorded eagerly is its own.)"""
    announce("backward while capturing")
    x = torch.randn(3, 100, device="cuda", requires_grad=True)
    ids = torch.zeros(3, 2, dtype=torch.int64, device="cuda")
    lp = ar.token_logprobs(x, ids[:, 0].contiguous()).logprob.sum()
    loss = ar.distill_loss(x, ids, torch.zeros(3, 2, device="cuda")).loss.sum()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    for y in (lp, loss):
        with pytest.raises(RuntimeError, match="captured"):
            y.backward()


@pytest.mark.parametrize("rows,cols,k", [(50, 200, 100), (300, 2000, 200), (300, 20000, 100), (4, 202048, 300)])
def test_distill_on_two_streams_and_captured(rows, cols, k):
    """distill_step with tables of ids: calls side by side, and replays on new teachers."""
    announce(f"distill streams [{rows},{cols}] k={k}")
    g = torch.Generator(device="cuda").manual_seed(k)
    xs = [torch.randn(rows, cols, device="cuda", generator=g).half() for _ in range(2)]
    ids = torch.randint(-1, min(cols, 3 * k), (rows, k), device="cuda", generator=g)
    v, w = torch.randn(rows, k, device="cuda", generator=g), torch.rand(rows, device="cuda", generator=g)

    def work(x):
        d = ar.distill_loss(x, ids, v)
        return [*ar.distill_step(x, ids, v, w), d.stats, ar.distill_loss_grad(x, ids, v, d.stats, w)]

    want = [work(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(work(xs[n]))
    torch.cuda.synchronize()
    for n in range(2):
        assert all(torch.equal(a, b) for outs in got[n] for a, b in zip(outs, want[n]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(xs[0])
    for n in range(3):
        ids.copy_(torch.randint(-1, min(cols, (n + 1) * k), (rows, k), device="cuda", generator=g))
        v.copy_(torch.randn(rows, k, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, work(xs[0]))), f"replay {n}"


def test_the_longest_row():
    """2^31 - 1 columns. At the temperature log2 e the exponents are the logits' differences, integers
    here, so that every term is a power of two or an integer times one and the lanes' sums (of 2^15
    terms) are exact; the merges of the 2^16 lanes' sums and of the slices round at most 24 times."""
    cols = 2 ** 31 - 1
    announce("longest row")
    t = float(np.float32(math.log2(math.e)))  # log2(e) / t rounds to 1
    x = torch.zeros(1, cols, dtype=torch.float16, device="cuda")
    spikes = {0: 20.0, 5: 21.0, 2 ** 30 + 3: 22.0, cols - 2: 21.0, cols - 1: 23.0}
    for at, value in spikes.items():
        x[0, at] = value
    best = sorted(spikes, key=lambda at: (-spikes[at], at)) + [1]
    total = (cols - len(spikes)) + sum(math.exp(s / t) for s in spikes.values())
    lse = math.log(total)
    lps = {at: spikes.get(at, 0.0) / t - lse for at in best + [7, 8, cols - 3]}
    entropy = lse - sum(math.exp(s / t) * s / t for s in spikes.values()) / total
    token = torch.tensor([cols - 1], device="cuda")
    r = ar.token_logprobs(x, token, temperature=t, entropy=True, top=6)
    # 24 roundings of the sum; the exponents, the logarithm and the last steps as in logits_reference
    # (|z| < 30); the entropy's quotient has twice the sum's roundings, times |z|
    tol, tol_entropy = R.U * (24 + 3 * 30 + 8 * 30), R.U * (2 * 24 * 30 + 3 * 30 + 8 * 30)
    assert r.top_tokens[0].tolist() == best
    for got, at in zip(r.top_logprobs[0].tolist(), best):
        assert abs(got - lps[at]) < tol
    assert abs(float(r.logprob) - lps[cols - 1]) < tol
    assert abs(float(r.entropy) - entropy) < tol_entropy
    w = torch.ones(1, device="cuda")
    grad = ar.token_logprobs_grad(x, token, r.stats, w, temperature=t)
    ids = torch.tensor([[cols - 1, 0, 7, cols - 1]], device="cuda")
    loss, dgrad = ar.distill_step(x, ids, torch.zeros(1, 4, device="cuda"), w, temperature=t)
    want = sum(0.25 * (math.log(0.25) - lps[at]) for at in ids[0].tolist())
    assert abs(float(loss) - want) < tol
    eps = torch.finfo(torch.float16).eps / 2
    q = {cols - 1: 0.5, 0: 0.25, 7: 0.25}
    for at, lp in lps.items():
        p = math.exp(lp)
        for got, exact in [(grad[0, at], ((at == cols - 1) - p) / t), (dgrad[0, at], (p - q.get(at, 0.0)) / t)]:
            # half a step of the type (2^-25 below its normal range), and the binary32 errors of p and q
            assert abs(float(got) - exact) <= abs(exact) * eps + 2.0 ** -25 + 2 * tol * (p + q.get(at, 0.0))


@pytest.mark.parametrize("dtype,top", [("f16", 64), ("f32", 1)])
def test_very_wide_rows_by_one_workgroup(capacity, dtype, top):
    """Rows far longer than a workgroup's registers and segments, left to one workgroup each."""
    capacity(2048)
    rows, cols = 2, 3_000_001
    announce(f"wide by one workgroup {dtype}")
    assert B.argreduce_logprobs_plan(rows, cols, dtype)["path"] == B.PATH_BLOCK
    rng = np.random.default_rng(41)
    x = torch.from_numpy(rng.normal(size=(rows, cols)) * 3).to(DT[dtype]).cuda()
    tokens = torch.tensor([cols - 1, 0], device="cuda")
    got = check_logprobs(x, tokens, dtype, 1.0, True, top)
    check_logprobs_grad(x, tokens, dtype, 1.0, True, *got, rng)
    check_distill(x, *make_teacher(rng, rows, cols, 300), dtype, 1.0, rng)


def test_calls_without_the_fast_module(monkeypatch):
    """The same bits through ctypes alone."""
    announce("ctypes")
    import argmin_reduction_wide_amd.logits as L
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(5, 60001, device="cuda", generator=g)
    tokens = torch.randint(0, 60001, (5,), device="cuda", generator=g)
    w = torch.rand(5, device="cuda", generator=g)

    def work():
        r = ar.token_logprobs(x, tokens, temperature=0.7, entropy=True, top=5)
        d = ar.distill_loss(x, r.top_tokens, r.top_logprobs, temperature=0.7)
        return [r.stats, r.top_logprobs, r.top_tokens, d.stats,
                ar.token_logprobs_grad(x, tokens, r.stats, w, w, temperature=0.7),
                ar.distill_loss_grad(x, r.top_tokens, r.top_logprobs, d.stats, w, temperature=0.7),
                *ar.distill_step(x, r.top_tokens, r.top_logprobs, w, temperature=0.7)]

    fast = work()

    class Ctypes:
        def __getattr__(self, name):
            return getattr(B.lib(), "argreduce_" + name)

    monkeypatch.setattr(L, "_call", Ctypes())
    for a, b in zip(fast, work()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rows,cols", [(5, 4), (5, 24), (5, 100), (5, 700), (5, 9000), (5, 140001)])
def test_an_id_beyond_an_empty_row(dtype, rows, cols):
    """A weight beyond the row makes loss and gradient NaN, also where every logit is -inf: by a group
    of lanes, a wavefront, a workgroup and split."""
    announce(f"beyond an empty row {dtype} [{rows},{cols}]")
    rng = np.random.default_rng(cols)
    x = torch.from_numpy(rng.normal(size=(rows, cols))).to(DT[dtype]).cuda()
    x[:3] = -INF
    ids = torch.tensor([[cols, 1], [1, cols + 7], [1, 2], [cols, 1], [2 ** 40, -1]], device="cuda")
    v = torch.zeros(rows, 2, device="cuda")
    v[3, 0] = -INF  # beyond the row, but without weight
    check_distill(x, ids, v, dtype, 1.0, rng)
    loss = ar.distill_loss(x, ids, v).loss
    assert loss.isnan().tolist() == [True, True, False, False, True] and loss[2] == INF


@pytest.mark.parametrize("rows,cols,step", [((1 << 26) + 5, 264, True), (1 << 28, 64, False)])
def test_more_rows_than_other_calls_hold(rows, cols, step):
    """A step of more rows than a launch holds wavefronts; a loss whose separate gradient call would
    not fit a launch."""
    announce(f"distill [{rows},{cols}] step={step}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.empty(rows, cols, dtype=torch.float16, device="cuda").normal_(generator=g)
    ids = torch.randint(0, cols, (rows, 1), device="cuda", generator=g)
    v, w = torch.zeros(rows, 1, device="cuda"), torch.ones(rows, device="cuda")
    if step:
        loss, grad = ar.distill_step(x, ids, v, w)
        with pytest.raises(ar.ArgreduceError):
            ar.distill_loss(x, ids, v)
    else:
        d = ar.distill_loss(x, ids, v)
        loss, grad = d.loss, None
        with pytest.raises(ar.ArgreduceError):
            ar.distill_loss_grad(x, ids, v, d.stats, w)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, rows // 2 - 1, rows // 3, (1 << 26) - 1, rows - 5, rows - 1], device="cuda")
    xs, i_s = host(x[at]), ids[at].cpu().numpy()
    for n in range(len(xs)):
        want = R.distill_row(xs[n], i_s[n], np.zeros(1), 1.0)
        R.agree(host(loss[at])[n], want["loss"], want["tol"], f"sample {n}")
        if step:
            d, tol = R.distill_grad_row(want, xs[n], 1.0, 1.0, "f16")
            R.agree(host(grad[at])[n], d, tol, f"sample {n} gradient")
    del x, ids, v, w, loss, grad
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rows,cols", [(13, 50), (13, 700), (13, 9000), (13, 140001), (3, 202048)])
def test_outputs_may_be_written_over(dtype, rows, cols):
    """The gradient does not depend on what a caller does with the log probabilities and entropies."""
    announce(f"outputs written over {dtype} [{rows},{cols}]")
    rng = np.random.default_rng(cols)
    x = make_rows(rng, rows, cols, dtype)
    tokens = make_tokens(rng, rows, cols)
    w, e = torch.ones(rows, device="cuda"), torch.ones(rows, device="cuda")
    for top in (0, 3):
        r = ar.token_logprobs(x, tokens, entropy=True, top=top)
        assert r.stats.shape == (4, rows)
        assert torch.equal(r.logprob.nan_to_num(9.0), r.stats[0].nan_to_num(9.0))
        assert torch.equal(r.entropy.nan_to_num(9.0), r.stats[1].nan_to_num(9.0))
        want = ar.token_logprobs_grad(x, tokens, r.stats, w, e)
        r.logprob.fill_(7.0)
        r.entropy.mul_(0.0)
        got = ar.token_logprobs_grad(x, tokens, r.stats, w, e)
        assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))
    ids, v = make_teacher(np.random.default_rng(1), rows, cols, 4)
    d = ar.distill_loss(x, ids, v)
    want = ar.distill_loss_grad(x, ids, v, d.stats, w)
    d.loss.fill_(7.0)
    got = ar.distill_loss_grad(x, ids, v, d.stats, w)
    assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))


ENTROPY_APART = 0x61706172  # as the header has it


@pytest.mark.parametrize("entropy", [0, 1, 2, -1, -2, 2 ** 31 - 1, ENTROPY_APART])
@pytest.mark.parametrize("rows,cols", [(3, 50), (3, 700), (3, 9000), (3, 202048)])
def test_rows_of_the_statistics(rows, cols, entropy):
    """[4, rows], and the entropy again in a fifth row for ARGREDUCE_ENTROPY_APART alone."""
    announce(f"statistics [{rows},{cols}] entropy={entropy}")
    x = torch.randn(rows, cols, device="cuda")
    tokens = torch.tensor([0, -1, cols - 1], device="cuda")
    need = B.argreduce_logprobs_scratch_bytes(rows, cols, B.F32)
    scratch = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    want = ar.token_logprobs(x, tokens, entropy=True).stats
    stats = torch.full((6, rows), 5.0, device="cuda")
    for call in (B.fast().argreduce_logprobs, B.lib().argreduce_logprobs):
        stats.fill_(5.0)
        assert call(x.data_ptr(), B.F32, rows, cols, cols, tokens.data_ptr(), 1.0, entropy, 0, stats.data_ptr(),
                    0, 0, scratch.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(stats[0], want[0]) and torch.equal(stats[2:4], want[2:4])
        assert torch.equal(stats[1], want[1]) if entropy else stats[1].isnan().all()
        assert torch.equal(stats[4], want[1]) if entropy == ENTROPY_APART else (stats[4] == 5).all()
        assert (stats[5] == 5).all()


def test_gradient_over_another_argument_is_refused():
    announce("overlap with other arguments")
    rows, cols, k = 4, 8, 3
    buf = torch.zeros(256, device="cuda")
    out = buf[16:16 + rows * cols].view(rows, cols)
    x = torch.randn(rows, cols, device="cuda")
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    ids, v, w = torch.zeros(rows, k, dtype=torch.int64, device="cuda"), torch.zeros(rows, k, device="cuda"), \
        torch.ones(rows, device="cuda")
    stats, dstats = ar.token_logprobs(x, t, entropy=True).stats, ar.distill_loss(x, ids, v).stats

    def inside(like, at):  # like's values in buf, from element `at`
        r = buf[at:at + like.numel() * like.element_size() // 4].view(like.dtype).view(like.shape)
        return r.copy_(like)

    calls = [(ar.token_logprobs_grad, dict(tokens=t, stats=stats, grad_logprob=w, grad_entropy=w)),
             (ar.distill_loss_grad, dict(teacher_tokens=ids, teacher_logits=v, stats=dstats, grad_loss=w)),
             (ar.distill_step, dict(teacher_tokens=ids, teacher_logits=v, weights=w))]
    for f, args in calls:
        for name, value in args.items():
            n = value.numel() * value.element_size() // 4
            for at in (16 - n + 2, 16 + rows * cols - 2):  # the last or first 8 bytes shared
                if at >= 0:
                    with pytest.raises(ValueError, match=f"overlap {name}"):
                        f(x, **{**args, name: inside(value, at)}, out=out)
            buf.fill_(5.0)
            f(x, **{**args, name: inside(value, 16 + rows * cols)}, out=out)  # right behind it
            assert not (out == 5).any()
    with pytest.raises(ValueError, match="overlap scratch"):
        ar.distill_step(x, ids, v, w, out=out, scratch=buf)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("cap,path", [(256 * 2048, B.PATH_SPLIT), (2048, B.PATH_BLOCK)])
@pytest.mark.parametrize("cols", [100001, 140001])
def test_special_rows_split_and_whole(capacity, dtype, cap, path, cols):
    """Rows of every kind, tokens and teacher entries beyond the row or absent, where the rows are
    split over workgroups and where a workgroup has one each. (The step of a 16-bit row of 100001 is
    one kernel, its loss alone is split.)"""
    rows = 13
    capacity(cap)
    for plan in (B.argreduce_logprobs_plan, B.argreduce_distill_plan):
        assert plan(rows, cols, dtype)["path"] == path
    announce(f"special rows {dtype} [{rows},{cols}] path {path}")
    rng = np.random.default_rng(cols)
    x = make_rows(rng, rows, cols, dtype)
    tokens = make_tokens(rng, rows, cols)
    kinds = set()
    for top in (0, 7, 64):
        got = check_logprobs(x, tokens, dtype, 1.3, top != 0, top)
        kinds |= {(row["kind"], row.get("beyond")) for row in got[3]}
    assert kinds == {("ok", False), ("ok", True), ("nan", None), ("empty", None), ("left out", None)}
    check_logprobs_grad(x, tokens, dtype, 1.3, True, *got, rng)
    for k in (1, 40, 300, 1024):
        ids, v = make_teacher(rng, rows, cols, k)
        v[8, 0] = 50.0                     # the id beyond the row has weight
        ids[0, 0], v[0, 0] = cols - 1, 9.0
        ids[7, 0], v[7, 0] = 5, INF        # a teacher of +inf
        ids[2, 0], v[2, 0] = 5, 1.0        # an empty row with a teacher
        ids[12] = ids[12, 0].clamp(min=0)  # one id, k times
        check_distill(x, ids, v, dtype, 1.3, rng)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("cols", [24, 700, 9000, 202048])
def test_gradient_at_masked_logits(dtype, cols):
    """A masked logit has the gradient of its own log probability and no other."""
    announce(f"masked logits {dtype} cols={cols}")
    x = torch.randn(2, cols, device="cuda").to(DT[dtype])
    x[:, 3:9] = -INF
    tokens = torch.tensor([5, 0], device="cuda")
    w, half = torch.full((2,), 3.0, device="cuda"), torch.full((2,), 0.5, device="cuda")
    r = ar.token_logprobs(x, tokens, temperature=2.0, entropy=True)
    assert r.logprob[0] == -INF and r.logprob[1].isfinite()
    g = ar.token_logprobs_grad(x, tokens, r.stats, w, half, temperature=2.0)
    near = 8 * R.U + R.HALF_STEP[dtype]  # the scale, the weight and the product, and the type's rounding
    assert abs(float(g[0, 5]) - 1.5) <= 1.5 * near and (g[0, 3:5] == 0).all() and (g[0, 6:9] == 0).all() and (g[1, 3:9] == 0).all()
    ids = torch.tensor([[5, 0], [0, 1]], device="cuda")
    loss, g = ar.distill_step(x, ids, torch.zeros(2, 2, device="cuda"), w, temperature=2.0)
    assert loss[0] == INF and loss[1].isfinite()
    assert abs(float(g[0, 5]) + 0.75) <= 0.75 * near and (g[0, 3:5] == 0).all() and (g[0, 6:9] == 0).all() and (g[1, 3:9] == 0).all()
