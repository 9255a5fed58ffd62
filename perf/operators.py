"""The logits operators as a program calls them: inputs, one pass, and the work it stands for.

Four kinds of pass over logits [rows, cols]:

* ``logprobs``        log probabilities of given tokens, entropy and top alternatives (scoring,
                      serving, writing down a teacher's top logits);
* ``logprobs_train``  the same log probabilities and entropy, and the gradient of a weighted
                      sum of them with respect to the logits (policy gradients);
* ``distill``         the distillation loss against a teacher's top logits (evaluation);
* ``distill_train``   that loss and its gradient (a training step's last layer).

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own``
true it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def _case(kind, rows, cols, dtype, pad=0, top=0, entropy=False, k=0, temperature=1.0, std=2.0,
          masked=0.0, skipped=0.0, **name):
    return dict(name, kind=kind, rows=rows, cols=cols, dtype=dtype, pad=pad, top=top, entropy=entropy,
                k=k, temperature=temperature, std=std, masked=masked, skipped=skipped)


def listed():
    return [
        # one sequence being decoded, a small vocabulary: the smallest call, latency only
        _case("logprobs", 1, 32000, "f32", top=5, entropy=True, name="score_1x32000_f32_top5"),
        # one sequence, sampler logits of a large vocabulary, with as many alternatives as APIs offer
        _case("logprobs", 1, 202048, "f32", top=20, entropy=True, temperature=0.7,
              name="score_1x202048_f32_top20"),
        # a decoding batch under a grammar: part of the vocabulary masked to -inf
        _case("logprobs", 32, 202048, "bf16", top=8, entropy=True, masked=0.3,
              name="score_32x202048_bf16_top8"),
        # scoring a prompt: one token per position, no alternatives; padded positions left out,
        # the vocabulary padded to a multiple of 64 in memory
        _case("logprobs", 4001, 32001, "f16", pad=63, skipped=0.1, name="score_4001x32001_f16"),
        # a small output alphabet, many positions: short rows
        _case("logprobs", 65536, 64, "f16", top=2, entropy=True, name="score_65536x64_f16_top2"),
        # a teacher writing down its top logits for later distillation
        _case("logprobs", 2048, 128256, "bf16", top=64, name="teacher_2048x128256_bf16_top64"),
        # policy gradient with an entropy bonus, a small microbatch of an odd vocabulary
        _case("logprobs_train", 257, 32003, "f32", entropy=True, skipped=0.25,
              name="policy_257x32003_f32"),
        # the same over a long batch
        _case("logprobs_train", 2048, 128256, "bf16", entropy=True, temperature=0.8,
              name="policy_2048x128256_bf16"),
        # evaluating a student on a held-out batch
        _case("distill", 512, 128256, "f16", k=32, name="distill_512x128256_f16_k32"),
        # the smallest training step: a handful of positions
        _case("distill_train", 16, 32000, "f32", k=8, temperature=2.0,
              name="distill_train_16x32000_f32_k8"),
        # odd sizes, rows padded in memory, positions without a teacher
        _case("distill_train", 1003, 50001, "f16", pad=15, k=33, skipped=0.1,
              name="distill_train_1003x50001_f16_k33"),
        # a training batch of a large vocabulary: the largest
        _case("distill_train", 4096, 128256, "bf16", k=64, name="distill_train_4096x128256_bf16_k64"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["logprobs", "logprobs_train", "distill", "distill_train"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    cols = _spread(rng, 16, 262144)
    train = kind.endswith("train")
    budget = 2 * 4096 * 128256 // ((2 if train else 1) * SIZE[dtype])  # elements, under the largest listed case
    rows = _spread(rng, 1, max(1, min(65536, 4 * budget // (5 * cols))))
    c = _case(kind, rows, cols, dtype, pad=rng.choice([0, 0, 0, rng.randrange(1, 64)]),
              temperature=rng.choice([1.0, 1.0, round(rng.uniform(0.5, 3.0), 2)]),
              std=round(rng.uniform(1.0, 4.0), 2), masked=rng.choice([0.0, 0.0, 0.2]),
              skipped=rng.choice([0.0, 0.0, 0.15]))
    if kind == "logprobs":
        c["top"] = rng.choice([0, _spread(rng, 1, max(1, min(64, cols // 4)))])
        if c["top"]:
            c["skipped"] = 0.0
    if not kind.startswith("distill"):
        c["entropy"] = rng.random() < 0.6
    else:
        c["k"] = _spread(rng, 1, min(256, cols))
        c["masked"] = 0.0
    return c


def _skipped(case):
    return int(case["rows"] * case["skipped"])


def prepare(case, seed):
    rows, cols, dtype, dev = case["rows"], case["cols"], DTYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(rows, cols + case["pad"], dtype=dtype, device=dev, generator=g)
    x = x.mul_(case["std"])[:, :cols]  # rows further apart than cols where there is padding
    left_out = torch.randperm(rows, device=dev, generator=g)[:_skipped(case)]
    s = {"kind": case["kind"], "logits": x, "temperature": case["temperature"], "top": case["top"],
         "entropy": case["entropy"]}
    if case["kind"].startswith("logprobs"):
        if case["masked"]:
            allowed = torch.rand(rows, cols, device=dev, generator=g) >= case["masked"]
            allowed[:, ::8] = True
            x.masked_fill_(~allowed, -math.inf)
        # the tokens that were sampled or given: mostly ones that the model finds likely
        tokens = torch.randint(0, cols, (rows,), device=dev, generator=g)
        liked = case["std"] * (2.5 + torch.randn(rows, 1, device=dev, generator=g))
        x.scatter_(1, tokens[:, None], liked.to(dtype))
        tokens[left_out] = -100
        s["tokens"] = tokens
        if case["kind"] == "logprobs_train":
            s["g_logprob"] = -torch.randn(rows, device=dev, generator=g).exp_()
            s["g_entropy"] = torch.full((rows,), -0.01, device=dev) if case["entropy"] else None
    else:
        k = case["k"]
        first = torch.randint(0, cols, (rows, 1), device=dev, generator=g)
        apart = torch.randint(1, cols // k + 1, (rows, 1), device=dev, generator=g)
        ids = (first + apart * torch.arange(k, device=dev)) % cols  # k different tokens
        v = 3.0 * torch.randn(rows, k, device=dev, generator=g) + 8.0
        v = v.sort(dim=1, descending=True).values
        noise = torch.randn(rows, k, device=dev, generator=g)
        x.scatter_(1, ids, (0.8 * v + noise).to(dtype))  # a student that half agrees
        # every third row's teacher has fewer alternatives: the rest of the row is empty
        fewer = (torch.arange(rows, device=dev) % 3 == 2)[:, None] & (torch.arange(k, device=dev) > k // 2)
        ids.masked_fill_(fewer, -1)
        v.masked_fill_(fewer, -math.inf)
        ids[left_out] = -1
        s.update(teacher_tokens=ids, teacher_logits=v)
        if case["kind"] == "distill_train":
            s["weights"] = torch.rand(rows, device=dev, generator=g) + 0.5
    return s


def _log_softmax(s):
    x = s["logits"].float() / s["temperature"]
    z = x - x.amax(dim=1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    return x, z - z.exp().sum(dim=1, keepdim=True).log()


def _top(x, logp, k):
    """The k largest of each row, ties to the lowest index: value and index as one integer."""
    order = (x + 0.0).view(torch.int32)
    order = order ^ ((order >> 31) & 0x7FFFFFFF)
    index = torch.arange(x.shape[1], device=x.device)
    tokens = 0xFFFFFFFF - (order.long() * (1 << 32) + (0xFFFFFFFF - index)).topk(k, dim=1).values % (1 << 32)
    return logp.gather(1, tokens), tokens


def _plain(s):
    x, logp = _log_softmax(s)
    if s["kind"].startswith("logprobs"):
        given = s["tokens"] >= 0
        at = s["tokens"].clamp(min=0)[:, None]
        lp = torch.where(given, logp.gather(1, at)[:, 0], 0.0)
        out = {"logprob": lp}
        if s["entropy"]:
            p = logp.exp()
            h = -torch.where(p > 0, p * logp, 0.0).sum(dim=1)
            out["entropy"] = torch.where(given, h, 0.0)
        if s["top"]:
            out["top_logprobs"], out["top_tokens"] = _top(s["logits"].float(), logp, s["top"])
        if s["kind"] == "logprobs_train":
            p = logp.exp()
            d = -p * s["g_logprob"][:, None]
            d.scatter_add_(1, at, s["g_logprob"][:, None])
            if s["entropy"]:
                d -= s["g_entropy"][:, None] * torch.where(p > 0, p * (logp + h[:, None]), 0.0)
            d = torch.where(given[:, None], d / s["temperature"], 0.0)
            out["grad"] = d.to(s["logits"].dtype)
        return out
    present = s["teacher_tokens"] >= 0
    ids = s["teacher_tokens"].clamp(min=0)
    some = present.any(dim=1, keepdim=True)
    v = torch.where(present, s["teacher_logits"], -math.inf) / s["temperature"]
    z = v - v.amax(dim=1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = z.exp()
    total = e.sum(dim=1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
    q = e / total
    away = torch.where(q > 0, q * (z - total.log() - logp.gather(1, ids)), 0.0)
    out = {"loss": away.sum(dim=1)}
    if s["kind"] == "distill_train":
        d = torch.where(some, logp.exp(), 0.0)
        d.scatter_add_(1, ids, -q)
        out["grad"] = (d * (s["weights"] / s["temperature"])[:, None]).to(s["logits"].dtype)
    return out


def _call(s):
    import argmin_reduction_wide_amd as ar

    x, t = s["logits"], s["temperature"]
    if s["kind"].startswith("logprobs"):
        r = ar.token_logprobs(x, s["tokens"], temperature=t, entropy=s["entropy"], top=s["top"])
        out = {"logprob": r.logprob}
        if s["entropy"]:
            out["entropy"] = r.entropy
        if s["top"]:
            out["top_logprobs"], out["top_tokens"] = r.top_logprobs, r.top_tokens
        if s["kind"] == "logprobs_train":
            out["grad"] = ar.token_logprobs_grad(x, s["tokens"], r.stats, s["g_logprob"], s["g_entropy"],
                                                 temperature=t)
        return out
    if s["kind"] == "distill_train":
        loss, grad = ar.distill_step(x, s["teacher_tokens"], s["teacher_logits"], s["weights"], temperature=t)
        return {"loss": loss, "grad": grad}
    return {"loss": ar.distill_loss(x, s["teacher_tokens"], s["teacher_logits"], temperature=t).loss}


def run(state):
    return _call(state) if own else _plain(state)


def work(case):
    rows, cols, size = case["rows"], case["cols"], SIZE[case["dtype"]]
    read = rows - _skipped(case)  # rows whose logits count
    n = read * cols
    if case["kind"].startswith("logprobs"):
        by = n * size + rows * (8 + 4 + 4 * case["entropy"] + 12 * case["top"])
        flops = n * (4 + 3 * case["entropy"])
        extra = rows * (4 + 4 * case["entropy"])
    else:
        by = n * size + rows * (12 * case["k"] + 4)
        flops = n * 4 + rows * case["k"] * 6
        extra = rows * 4
    if case["kind"].endswith("train"):
        by += rows * cols * size + extra
        flops += n * (4 + 3 * case["entropy"])
    return {"bytes": by, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    parts = []
    step = max(1, (1 << 27) // case["cols"])
    for a in range(0, case["rows"], step):
        cut = {k: v[a:a + step] if torch.is_tensor(v) else v for k, v in s.items()}
        parts.append(_exact_rows(cut))
    return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_rows(s):
    t = s["temperature"]
    y = s["logits"].double() / t
    norm = torch.logsumexp(y, dim=1)
    p = torch.softmax(y, dim=1)
    rows = torch.arange(y.shape[0], device=y.device)
    out = {}
    if s["kind"].startswith("logprobs"):
        live = (s["tokens"] >= 0).double()
        j = torch.where(s["tokens"] >= 0, s["tokens"], 0)
        out["logprob"] = torch.where(live > 0, y[rows, j] - norm, 0.0)
        if s["entropy"]:
            mean = torch.where(p > 0, p * y, 0.0).sum(dim=1)
            out["entropy"] = live * (norm - mean)
        if s["top"]:
            out["top_logprobs"] = y.topk(s["top"], dim=1).values - norm[:, None]
            out["top_tokens"] = None
        if s["kind"] == "logprobs_train":
            a = live * s["g_logprob"].double() / t
            grad = -a[:, None] * p
            grad[rows, j] += a
            if s["entropy"]:
                b = live * s["g_entropy"].double() / t
                grad -= b[:, None] * torch.where(p > 0, p * (y - mean[:, None]), 0.0)
            out["grad"] = grad
        return out
    there = s["teacher_tokens"] >= 0
    q = torch.where(there, (s["teacher_logits"].double() / t).exp(), 0.0)
    some = there.any(dim=1)
    q = q / torch.where(some, q.sum(dim=1), 1.0)[:, None]
    j = torch.where(there, s["teacher_tokens"], 0)
    logp = y[rows[:, None], j] - norm[:, None]
    out["loss"] = (torch.special.xlogy(q, q) - torch.where(q > 0, q * logp, 0.0)).sum(dim=1)
    if s["kind"] == "distill_train":
        grad = p * some[:, None]
        grad.index_put_((rows[:, None].expand_as(j), j), -q, accumulate=True)
        out["grad"] = grad * (s["weights"].double() / t)[:, None]
    return out
