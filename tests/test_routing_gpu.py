"""Expert routing on the GPU against the plain 64-bit reference (choices_reference.py): special rows, ties, layouts,
streams, graphs, autograd and a training step."""
import math

import numpy as np
import pytest
import torch

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B
import choices_reference as C
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


def make_logits(rng, groups, tokens, experts, dtype, nan=False):
    x = rng.normal(size=(groups, tokens, experts)) * 2
    low = torch.finfo(DT[dtype]).min
    for t in range(tokens):
        kind = t % 9
        if kind == 1:
            x[:, t, rng.random(experts) < 0.5] = -INF
        elif kind == 2:
            x[:, t] = -INF
        elif kind == 3:
            x[:, t] = 0.5
        elif kind == 4:
            x[:, t] = low
        elif kind == 5:
            x[:, t, rng.random(experts) < 0.5] = low
        elif kind == 6:
            x[:, t] = rng.integers(0, 3, size=experts)
        elif kind == 7:
            x[:, t, 0::2] = 0.0
            x[:, t, 1::2] = -0.0
    if nan and tokens > 4:
        x[0, 4, int(rng.integers(experts))] = math.nan
        if groups > 2:
            x[2, 0, int(rng.integers(experts))] = INF
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def check(x, top, dtype, live=None, renormalize=False, rng=None):
    """A call and its gradient against the reference, group by group."""
    r = ar.route_experts(x, top, live=live, renormalize=renormalize)
    lead, (tokens, experts) = x.shape[:-2], x.shape[-2:]
    rng = rng or np.random.default_rng(0)
    gw = torch.from_numpy(rng.normal(size=(*lead, tokens, top))).float().cuda()
    gb = torch.from_numpy(rng.normal(size=lead)).float().cuda()
    gz = torch.from_numpy(rng.normal(size=lead)).float().cuda()
    grad = ar.route_experts_grad(x, r, gw, gb, gz, live=live, renormalize=renormalize)
    torch.cuda.synchronize()
    assert grad.dtype == x.dtype and grad.shape == x.shape and grad.is_contiguous()
    assert r.weights.shape == r.experts.shape == (*lead, tokens, top) and r.counts.shape == (*lead, experts)
    xs = host(x).reshape(-1, tokens, experts)
    ls = np.ones(xs.shape[:2], bool) if live is None else live.cpu().numpy().reshape(xs.shape[:2])
    flat = lambda t, *s: host(t).reshape(-1, *s)  # noqa: E731
    w, e, c = flat(r.weights, tokens, top), flat(r.experts, tokens, top), flat(r.counts, experts)
    n, balance, z = flat(r.tokens), flat(r.balance), flat(r.z)
    gws, gbs, gzs, d = flat(gw, tokens, top), flat(gb), flat(gz), flat(grad, tokens, experts)
    for g in range(len(xs)):
        want = C.route_group(xs[g], ls[g], top, renormalize)
        what = f"group {g}"
        assert np.array_equal(e[g], want["experts"]), what
        assert np.array_equal(c[g], want["counts"]) and n[g] == want["n"], what
        R.agree(w[g], want["weights"], want["tol_w"], what + " weights")
        R.agree(balance[g], want["balance"], want["tol_balance"], what + " balance")
        R.agree(z[g], want["z"], want["tol_z"], what + " z")
        for t in range(tokens):
            dw, tol = C.route_grad_token(want, t, renormalize, gws[g, t], gbs[g], gzs[g], dtype)
            R.agree(d[g, t], dw, tol, f"{what} token {t} gradient")
    return r


EXPERTS = [1, 2, 3, 7, 8, 9, 16, 31, 64, 65, 100, 128, 129, 255, 256, 257, 500, 512, 513, 1000, 1024]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("experts", EXPERTS)
def test_route_and_gradient(dtype, experts):
    rng = np.random.default_rng(experts)
    for top in sorted({1, min(2, experts), min(8, experts), min(64, experts)}):
        renormalize = bool((top + experts) % 2)
        announce(f"route {dtype} experts={experts} top={top} renormalize={renormalize}")
        x = make_logits(rng, 3, 19, experts, dtype, nan=top == 1)
        live = torch.from_numpy(rng.random((3, 19)) < 0.8).cuda()
        check(x, top, dtype, live, renormalize, rng)
        check(x[:1], top, dtype, None, not renormalize, rng)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("experts", [9, 16, 17, 33, 64, 127, 256, 300, 512, 1000])
def test_nine_and_more_choices(dtype, experts):
    """Lists of up to sixteen and, above that, choices taken one by one; rows with fewer logits than choices."""
    rng = np.random.default_rng(experts + 5)
    for top in sorted({9, min(15, experts), min(16, experts), min(17, experts)}):
        announce(f"route {dtype} experts={experts} top={top}")
        x = make_logits(rng, 2, 21, experts, dtype)
        x[0, 3:6, 5:] = -INF
        check(x, top, dtype, None, top % 2 == 0, rng)


@pytest.mark.parametrize("cap", [2048, 256 * 2048])
@pytest.mark.parametrize("tokens", [1, 2, 63, 700])
def test_tokens_over_workgroups(capacity, cap, tokens):
    capacity(cap)
    rng = np.random.default_rng(tokens)
    for dtype, experts, top in (("bf16", 24, 3), ("f32", 130, 9)):
        announce(f"route {dtype} tokens={tokens} experts={experts} capacity {cap}")
        check(make_logits(rng, 2, tokens, experts, dtype), top, dtype, None, True, rng)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("offset", [1, 3, 5])
@pytest.mark.parametrize("experts,pad", [(10, 6), (64, 0), (64, 1), (100, 3), (515, 8)])
def test_strides_and_alignment(dtype, offset, experts, pad):
    groups, tokens = 2, 21
    rng = np.random.default_rng(offset * experts)
    announce(f"route strides {dtype} experts={experts} pad={pad} offset={offset}")
    rows = groups * tokens
    buf = torch.full((rows * (experts + pad) + offset + 16,), math.nan, dtype=DT[dtype], device="cuda")
    x = buf[offset:offset + rows * (experts + pad)].view(groups, tokens, experts + pad)[..., :experts]
    x.copy_(make_logits(rng, groups, tokens, experts, dtype))
    r = check(x, 4, dtype, None, True, rng)
    # a gradient buffer at any element's address
    out = torch.full((rows * experts + offset + 8,), 7.0, dtype=DT[dtype], device="cuda")
    view = out[offset:offset + rows * experts].view(groups, tokens, experts)
    gw = torch.ones(groups, tokens, 4, device="cuda")
    gw[..., 0] = -1.0
    want = ar.route_experts_grad(x, r, gw, renormalize=True)
    assert ar.route_experts_grad(x, r, gw, renormalize=True, out=view) is view
    assert torch.equal(view, want)
    assert (out[:offset] == 7).all() and (out[offset + rows * experts:] == 7).all()


def test_leading_dimensions():
    announce("route leading dimensions")
    rng = np.random.default_rng(4)
    x = make_logits(rng, 6, 10, 12, "f32")
    r = check(x.view(2, 3, 10, 12), 3, "f32")
    assert r.balance.shape == (2, 3) and r.tokens.shape == (2, 3)
    one = check(x[0], 3, "f32")
    assert one.balance.shape == () and one.counts.shape == (12,)
    assert torch.equal(one.weights, r.weights[0, 0])
    none = ar.route_experts(x[:0], 3)
    assert none.weights.shape == (0, 10, 3) and none.balance.shape == (0,)
    empty = ar.route_experts(x[:, :0], 3)
    assert (empty.counts == 0).all() and (empty.balance == 0).all() and (empty.tokens == 0).all() and (empty.z == 0).all()
    assert ar.route_experts_grad(x[:, :0], empty, None, empty.balance).shape == (6, 0, 12)


def test_tokens_left_out():
    """Their logits may be anything; a group without tokens has losses 0."""
    announce("route tokens left out")
    x = torch.randn(3, 8, 20, device="cuda")
    live = torch.ones(3, 8, dtype=torch.bool, device="cuda")
    live[0, ::2] = False
    live[1] = False
    want = ar.route_experts(x, 2, live=live)
    y = x.clone()
    y[~live] = math.nan
    got = ar.route_experts(y, 2, live=live)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert (got.experts[~live] == -1).all() and (got.weights[~live] == 0).all()
    assert got.tokens.tolist() == [4, 0, 8] and got.balance[1] == 0 and got.z[1] == 0
    g = torch.ones(3, device="cuda")
    grad = ar.route_experts_grad(y, got, None, g, g, live=live)
    assert (grad[~live] == 0).all() and torch.equal(grad, ar.route_experts_grad(x, want, None, g, g, live=live))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("groups,tokens,experts,top", [(1, 60000, 64, 6), (7, 3001, 256, 8), (40, 1000, 17, 2)])
def test_many_tokens(dtype, groups, tokens, experts, top):
    """Whole batches against 64-bit torch, a sample of tokens against the reference and its bounds."""
    announce(f"route {dtype} [{groups},{tokens},{experts}] top {top}")
    g = torch.Generator(device="cuda").manual_seed(experts)
    x = (torch.randn(groups, tokens, experts, device="cuda", generator=g) * 1.5).to(DT[dtype])
    r = ar.route_experts(x, top)
    at = x.float().sort(dim=-1, descending=True, stable=True).indices[..., :top]
    assert torch.equal(r.experts, at)
    counts = torch.zeros(groups, experts, dtype=torch.int64, device="cuda")
    counts.scatter_add_(1, at.flatten(1), torch.ones_like(at).flatten(1))
    assert torch.equal(r.counts, counts) and (r.tokens == tokens).all()
    p = torch.softmax(x.double(), -1)
    balance = experts / (top * tokens ** 2) * (counts * p.sum(1)).sum(1)
    z = torch.logsumexp(x.double(), -1).square().mean(1)
    # p off by at most 3 E|z| + 3 |z| / ln 2 + adds + 14 < 200 u, sums of one sign by tokens u
    assert ((r.balance - balance).abs() / balance).max() < C.U * (200 + tokens + 600)
    assert ((r.z - z).abs() / z).max() < C.U * (400 + tokens + 600)
    assert ((r.weights - p.gather(-1, at)).abs() / p.gather(-1, at)).max() < C.U * 200


def test_offsets_beyond_32_bits():
    stride, experts = 2 ** 29 + 8, 24
    announce("route offsets beyond 32 bits")
    buf = torch.empty(9 * stride + experts, dtype=torch.float16, device="cuda")
    x = buf.as_strided((2, 5, experts), (5 * stride, stride, 1))
    rng = np.random.default_rng(3)
    x.copy_(torch.from_numpy(rng.normal(size=(2, 5, experts))).half().cuda())
    r = ar.route_experts(x, 3)
    y = x.contiguous()
    want = ar.route_experts(y, 3)
    for a, b in zip(r, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("soff", [0, 1, 13])
def test_scratch_and_output_bounds(soff):
    announce(f"route bounds offset {soff}")
    for groups, tokens, experts, top in ((3, 50, 10, 3), (2, 700, 130, 8)):
        x = torch.randn(groups, tokens, experts, device="cuda")
        want = ar.route_experts(x, top)
        need = B.argreduce_route_scratch_bytes(groups, tokens, experts, "f32")
        n = B.argreduce_route_totals_bytes(groups, experts)
        k = groups * tokens * top
        for fill in (0, 255, 90):
            scratch = torch.full((need + soff + 64,), fill, dtype=torch.uint8, device="cuda")
            totals = torch.full((n + 64,), 77, dtype=torch.uint8, device="cuda")
            w, e = torch.full((k + 16,), 7.0, device="cuda"), torch.full((k + 16,), 7, device="cuda")
            rc = B.argreduce_route(x.data_ptr(), "f32", groups, tokens, experts, experts, 0, top, 0, w.data_ptr(),
                                   e.data_ptr(), totals.data_ptr(), scratch.data_ptr() + soff, need,
                                   torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert rc == 0 and (totals[n:] == 77).all() and (w[k:] == 7).all() and (e[k:] == 7).all()
            assert (scratch[:soff] == fill).all() and (scratch[soff + need:] == fill).all()
            assert torch.equal(totals[:n].view(torch.int64), want.totals)
            assert torch.equal(w[:k], want.weights.flatten()) and torch.equal(e[:k], want.experts.flatten())


@pytest.mark.parametrize("groups,tokens,experts,top", [(1, 32, 256, 8), (16, 1000, 64, 2), (3, 5000, 513, 4)])
def test_same_bits_streams_and_graphs(groups, tokens, experts, top):
    announce(f"route [{groups},{tokens},{experts}] repeated, on two streams, captured")
    gen = torch.Generator(device="cuda").manual_seed(experts)
    xs = [torch.randn(groups, tokens, experts, device="cuda", generator=gen) for _ in range(2)]
    gw = torch.randn(groups, tokens, top, device="cuda", generator=gen)
    gb = torch.ones(groups, device="cuda")

    def both(x):
        r = ar.route_experts(x, top, renormalize=True)
        return (*r, ar.route_experts_grad(x, r, gw, gb, gb, renormalize=True))

    same = lambda a, b: all(torch.equal(u, v) for u, v in zip(a, b))  # noqa: E731
    want = [both(x) for x in xs]
    for _ in range(5):
        assert same(both(xs[0]), want[0])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(10):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(both(xs[k]))
    torch.cuda.synchronize()
    assert all(same(r, want[k]) for k in range(2) for r in got[k])
    x, graphs = xs[0].clone(), []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = both(x)
        graphs.append((graph, r))
    for i in range(6):
        x.copy_(xs[i % 2])
        both(xs[1])
        graphs[i % 2][0].replay()
        torch.cuda.synchronize()
        assert same(graphs[i % 2][1], want[i % 2])


def test_parts_of_the_gradient():
    """Each of the three gradients alone, and their sum; broadcast ones through autograd."""
    announce("route gradients alone")
    x = torch.randn(2, 30, 40, device="cuda")
    r = ar.route_experts(x, 4)
    gw, gb, gz = torch.randn(2, 30, 4, device="cuda"), torch.randn(2, device="cuda"), torch.randn(2, device="cuda")
    parts = [ar.route_experts_grad(x, r, gw), ar.route_experts_grad(x, r, None, gb),
             ar.route_experts_grad(x, r, None, None, gz)]
    whole = ar.route_experts_grad(x, r, gw, gb, gz)
    # three sums of up to 3 terms each, rounded once or thrice
    assert (whole - sum(parts)).abs().max() < 2.0 ** -20 * sum(p.abs().max() for p in parts)
    assert (ar.route_experts_grad(x, r) == 0).all()


@pytest.mark.parametrize("renormalize", [False, True])
def test_autograd(renormalize):
    announce(f"route autograd renormalize={renormalize}")
    x = torch.randn(2, 30, 40, device="cuda", requires_grad=True)
    live = torch.rand(2, 30, device="cuda") < 0.8
    r = ar.route_experts(x, 4, live=live, renormalize=renormalize)
    gw = torch.randn(2, 30, 4, device="cuda")
    loss = (r.weights * gw).sum() + 0.3 * r.balance.sum() + 0.1 * r.z.mean()
    for t in (r.experts, r.counts, r.tokens):
        assert not t.requires_grad
        t.zero_()                       # outputs of their own
    loss.backward()
    p = ar.route_experts(x.detach(), 4, live=live, renormalize=renormalize)
    want = ar.route_experts_grad(x.detach(), p, gw, torch.full((2,), 0.3, device="cuda"),
                                 torch.full((2,), 0.05, device="cuda"), live=live, renormalize=renormalize)
    assert (x.grad - want).abs().max() <= 2.0 ** -22 * want.abs().max()
    # one output alone
    x.grad = None
    ar.route_experts(x, 4, live=live, renormalize=renormalize).balance.sum().backward()
    want = ar.route_experts_grad(x.detach(), p, None, torch.ones(2, device="cuda"), live=live, renormalize=renormalize)
    assert torch.equal(x.grad, want)
    x.grad = None
    ar.route_experts(x, 4, renormalize=renormalize).weights.sum().backward()  # an expanded gradient
    assert torch.isfinite(x.grad).all()


@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_is_the_difference(renormalize):
    """Against central differences in 64 bits, the choice held fixed."""
    announce("route gradient against differences")
    rng = np.random.default_rng(8)
    x = rng.normal(size=(6, 9))
    t = torch.from_numpy(x).float().cuda()
    r = ar.route_experts(t, 3, renormalize=renormalize)
    gw, gb, gz = rng.normal(size=(6, 3)), 0.6, -0.2
    got = host(ar.route_experts_grad(t, r, torch.from_numpy(gw).float().cuda(), torch.tensor(gb, device="cuda"),
                                     torch.tensor(gz, device="cuda"), renormalize=renormalize))
    at, counts = r.experts.cpu().numpy(), r.counts.cpu().numpy()
    x = host(t)
    gw = host(torch.from_numpy(gw).float())

    def target(v):
        p = np.exp(v - v.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        w = np.take_along_axis(p, at, 1)
        if renormalize:
            w = w / w.sum(1, keepdims=True)
        lse = np.log(np.exp(v).sum(1))
        return (gw * w).sum() + gb * 9 / (3 * 36) * (counts * p.sum(0)).sum() + gz * (lse ** 2).mean()

    h = 1e-5
    for i in range(6):
        for j in range(9):
            up, down = x.copy(), x.copy()
            up[i, j] += h
            down[i, j] -= h
            # differences are good to h^2 and 1e-16 / h times the target's size, the kernel to 100 u
            assert abs((target(up) - target(down)) / (2 * h) - got[i, j]) < 1e-8 + 100 * C.U * 4


def test_captured_autograd_is_refused():
    announce("route autograd in a capture")
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    ar.route_experts(x, 2).balance.backward()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    refused = False
    with torch.cuda.graph(graph, stream=s):
        y = x.detach() * 2
        try:
            ar.route_experts(x, 2)
        except RuntimeError as e:
            refused = "captured" in str(e)
    torch.cuda.synchronize()
    assert refused and y is not None


def test_refusals():
    announce("route refusals")
    x = torch.zeros(2, 6, 16, device="cuda")
    live = torch.ones(2, 6, dtype=torch.bool, device="cuda")
    for logits, top, kw in [(x.double(), 2, {}), (x[..., ::2], 2, {}), (x, 0, {}), (x, 17, {}), (x[0, 0], 2, {}),
                            (x, 2, dict(live=live.byte())), (x, 2, dict(live=live[:1])), (x, 2, dict(live=live.cpu())),
                            (torch.zeros(2, 1025, device="cuda"), 2, {}), (torch.zeros(2, 100, device="cuda"), 65, {}),
                            (x.transpose(0, 1), 2, {}), (x[..., :0], 1, {}),
                            (x, 2, dict(scratch=torch.zeros(8, dtype=torch.uint8)))]:
        with pytest.raises((ValueError, ar.ArgreduceError)):
            ar.route_experts(logits, top, **kw)
    r = ar.route_experts(x, 2)
    gw, gb = torch.zeros(2, 6, 2, device="cuda"), torch.zeros(2, device="cuda")
    for args, kw in [((gw[..., :1],), {}), ((gw.double(),), {}), ((None, gb[:1]), {}), ((None, None, gb.cpu()), {}),
                     ((gw,), dict(out=torch.zeros(2, 6, 15, device="cuda"))), ((gw,), dict(out=x)),
                     ((gw,), dict(out=x.half())), ((gw,), dict(live=live[:1]))]:
        with pytest.raises(ValueError):
            ar.route_experts_grad(x, r, *args, **kw)
    with pytest.raises(ValueError):
        ar.route_experts_grad(x, r._replace(totals=r.totals[:-1]), gw)
    with pytest.raises(ValueError):
        ar.route_experts_grad(x, r._replace(experts=r.experts.int()), gw)
    big = torch.zeros(2 * 6 * 16 + 24, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        ar.route_experts_grad(x, r, big[:24].view(2, 6, 2), out=big[12:12 + 192].view(2, 6, 16))
    torch.cuda.synchronize()


def test_gradient_over_the_mask_is_refused():
    announce("route gradient over the mask")
    room = torch.zeros(4 * 192 + 12, dtype=torch.uint8, device="cuda")
    live, out = room[760:772].view(torch.bool).view(2, 6), room[:768].view(torch.float32).view(2, 6, 16)
    x = torch.randn(2, 6, 16, device="cuda")
    live.fill_(True)
    r = ar.route_experts(x, 2, live=live)
    with pytest.raises(ValueError, match="out must not overlap live"):
        ar.route_experts_grad(x, r, r.weights, live=live, out=out)
    torch.cuda.synchronize()


def test_weights_may_be_written_over():
    """What a caller writes into a result changes nothing that the gradient reads."""
    announce("route results written over")
    x = torch.randn(3, 7, 16, device="cuda")
    g = torch.randn(3, 7, 4, device="cuda")

    def work(write):
        y = x.clone().requires_grad_()
        r = ar.route_experts(y, 4)
        loss = (r.weights * g).sum() + r.balance.sum() + r.z.sum()
        if write:
            for t in (r.experts, r.counts, r.tokens):
                t.fill_(-7)
            with torch.no_grad():
                r.weights.fill_(9.0)
        loss.backward()
        return y.grad

    want = work(False)
    assert torch.equal(work(True), want)
    r = ar.route_experts(x, 4)
    r.weights.fill_(9.0)
    one = torch.ones(3, device="cuda")
    assert torch.equal(ar.route_experts_grad(x, r, g, one, one), want)


def test_calls_without_the_fast_module(monkeypatch):
    """The same bits through ctypes alone."""
    announce("ctypes")
    import argmin_reduction_wide_amd.routing as module
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(3, 501, 60, device="cuda", generator=g)
    w, v = torch.rand(3, 501, 6, device="cuda", generator=g), torch.rand(3, device="cuda", generator=g)
    live = torch.rand(3, 501, device="cuda", generator=g) < 0.9

    def work():
        r = ar.route_experts(x, 6, live=live, renormalize=True)
        return [*r, ar.route_experts_grad(x, r, w, v, v, live=live, renormalize=True)]

    fast = work()

    class Ctypes:
        def __getattr__(self, name):
            return getattr(B.lib(), "argreduce_" + name)

    monkeypatch.setattr(module, "_call", Ctypes())
    for a, b in zip(fast, work()):
        assert torch.equal(a, b)


def test_expert_numbers_beyond_the_row():
    """Bad numbers in what is passed back make no access out of range."""
    announce("route bad experts")
    x = torch.randn(2, 6, 16, device="cuda")
    r = ar.route_experts(x, 3)
    bad = r.experts.clone()
    bad[0, 0] = torch.tensor([16, 2 ** 40, -5])
    gw = torch.ones(2, 6, 3, device="cuda")
    got = ar.route_experts_grad(x, r._replace(experts=bad), gw)
    want = ar.route_experts_grad(x, r, gw)
    assert torch.equal(got[0, 1:], want[0, 1:]) and torch.equal(got[1], want[1])
    assert (got[0, 0] == 0).all()


def test_training_step():
    """A router trained on its losses alone: a step against the gradient moves both down, and autograd's step is the
    plain calls' step."""
    announce("route training step")
    g = torch.Generator(device="cuda").manual_seed(0)
    hidden = torch.randn(2, 200, 32, device="cuda", generator=g)
    w = torch.randn(32, 16, device="cuda", generator=g).requires_grad_()
    x = hidden @ w
    r = ar.route_experts(x, 2, renormalize=True)
    (r.balance.mean() + 0.01 * r.z.mean()).backward()
    plain = ar.route_experts(x.detach(), 2, renormalize=True)
    half, z = torch.full((2,), 0.5, device="cuda"), torch.full((2,), 0.005, device="cuda")
    dx = ar.route_experts_grad(x.detach(), plain, None, half, z, renormalize=True)
    want = hidden.flatten(0, 1).t().double() @ dx.flatten(0, 1).double()
    # sums of 400 products in 32 bits
    size = hidden.flatten(0, 1).t().abs().double() @ dx.flatten(0, 1).abs().double()
    assert ((w.grad.double() - want).abs() <= 500 * C.U * size + 1e-12).all()
