"""The operators over rows of vocabulary logits, as measured cases.

``run`` makes one pass through an operator: as a user calls it through
``pmm_fc_layer_gb300`` where ``own`` is true, else in plain torch operations
(32-bit arithmetic, one rounding at the end).  ``exact`` gives the same
outputs from the definition in 64 bits.  The operators, with z = logits / tau
and p = softmax(z) of a row:

logprobs      ln p[token], the entropy - sum p ln p, the logsumexp, and the k
              largest logits of the row (ties to the lowest index) with their
              ln p, best first
logprobs_bwd  dlogits = (g (onehot(token) - p) - h p (ln p + H)) / tau for
              gradients g of ln p[token] and h of the entropy H
distill       a teacher's list of k logits a row, q = softmax(list / tau):
              tau^2 KL(q | p) of each row, its mean over the counted rows, and
              the mean's gradient tau (p - q) / n

A row with keep = 0 counts for nothing: its outputs are zeros (indices -1).  A
token outside the vocabulary has ln p = 0 and no gradient; a list ends at its
first index outside the vocabulary, and an empty one leaves its row out.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


def _row(op, name, T, V, k=0, f32=False, tau=1.0, kept=1.0, entropy=False, allowed=1.0, grad=True,
         ragged=False):
    return {"name": name, "op": op, "T": T, "V": V, "k": k, "f32": f32, "tau": tau, "kept": kept,
            "entropy": entropy, "allowed": allowed, "grad": grad, "ragged": ragged}


def listed():
    return [
        # scoring a batch of sampled sequences for a policy step: ln p and entropy of every token
        _row("logprobs", "score_policy", 8192, 128256, entropy=True),
        # a teacher's pass: the lists that its students learn from
        _row("logprobs", "teacher_top64", 4096, 128256, k=64),
        # answering one token with its twenty alternatives
        _row("logprobs", "answer_one_top20", 1, 128256, k=20),
        # a decoding batch, sampled at a temperature, of which a grammar allows one word in twenty
        _row("logprobs", "answer_batch_grammar", 64, 128256, k=5, f32=True, tau=0.7, allowed=0.05),
        # an odd vocabulary in fp32, half of the positions masked
        _row("logprobs", "score_odd_f32_masked", 1003, 50257, k=1, f32=True, kept=0.5, entropy=True),
        # the way back of a policy step with its entropy bonus
        _row("logprobs_bwd", "policy_bwd", 8192, 128256, entropy=True),
        # the same for a ragged batch, fp32, padding and masked positions, no bonus
        _row("logprobs_bwd", "policy_bwd_odd_f32", 1003, 50257, f32=True, tau=0.7, kept=0.5),
        # a student's training step on lists of 64
        _row("distill", "distill_train", 4096, 128256, k=64, tau=2.0),
        # long lists cut where the teacher's probability is used up, an odd vocabulary in fp32, masked
        _row("distill", "distill_odd_f32_ragged", 777, 50257, k=100, f32=True, kept=0.5, ragged=True),
        # how far a student is from its teacher: the loss alone, on a validation batch
        _row("distill", "distill_loss_only", 1024, 50304, k=20, grad=False),
        # a few short positions over a small vocabulary: what a call costs
        _row("distill", "distill_small", 16, 1003, k=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_bwd", "distill"])
    f32 = rng.random() < 0.35
    while True:
        T, V = _log(rng, 1, 8192), _log(rng, 500, 262144)
        if T * V * (2 if f32 else 1) <= 8192 * 128256:
            break
    c = _row(op, "", T, V, f32=f32, tau=rng.choice([1.0, 1.0, 0.7, 2.0]),
             kept=rng.choice([1.0, 0.9, 0.5]))
    del c["name"]
    if op != "distill":
        c["entropy"] = rng.random() < 0.5
        c["allowed"] = rng.choice([1.0, 1.0, 0.25])
        c["k"] = rng.choice([0, _log(rng, 1, 64), _log(rng, 1, 128)]) if op == "logprobs" else 0
        if c["k"] * 8 > V:
            c["allowed"] = 1.0
    else:
        c["k"] = _log(rng, 1, 256)
        c["grad"] = rng.random() < 0.75
        c["ragged"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _space(rows, cols, dtype):
    ld = (cols + 7) // 8 * 8
    return torch.empty((rows, ld), device="cuda", dtype=dtype)[:, :cols]


def _chunks(T, V, most=1 << 28):
    step = max(1, most // V)
    return [(r, min(T, r + step)) for r in range(0, T, step)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T, V, k = case["op"], case["T"], case["V"], case["k"]
    dtype = F32 if case["f32"] else BF16
    s = {"case": case, "logits": _space(T, V, dtype)}
    tokens = torch.randint(0, V, (T,), device="cuda", generator=g)
    # rows from undecided to nearly certain
    spread = torch.rand((T, 1), device="cuda", generator=g).mul_(2.5).add_(0.8)
    lift = torch.rand(T, device="cuda", generator=g).mul_(14)
    if op == "distill":
        s["top_index"] = torch.empty((T, k), device="cuda", dtype=torch.int32)
        s["top_logit"] = torch.empty((T, k), device="cuda")
    for a, b in _chunks(T, V):
        z = torch.randn((b - a, V), device="cuda", generator=g).mul_(spread[a:b])
        rows = torch.arange(b - a, device="cuda")
        if case["allowed"] < 1:
            z.masked_fill_(torch.rand((b - a, V), device="cuda", generator=g) >= case["allowed"], -math.inf)
            z[rows, tokens[a:b]] = 0.0
        z[rows, tokens[a:b]] += lift[a:b]
        s["logits"][a:b] = z
        if op == "distill":  # a teacher whose logits are near the student's
            z.add_(torch.randn((b - a, V), device="cuda", generator=g), alpha=0.5)
            best = z.topk(k, dim=1)
            s["top_index"][a:b], s["top_logit"][a:b] = best.indices, best.values
    s["keep"] = None
    if case["kept"] < 1:
        s["keep"] = (torch.rand(T, device="cuda", generator=g) < case["kept"]).to(torch.uint8)
    f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
    if op == "distill":
        if case["ragged"]:
            length = torch.randint(1, k + 1, (T, 1), device="cuda", generator=g)
            s["top_index"].masked_fill_(torch.arange(k, device="cuda") >= length, -1)
        s["token_loss"], s["loss"] = torch.empty(T, **f32), torch.empty(1, **f32)
        s["kept"] = torch.empty(1, **i32)
        s["dlogits"] = _space(T, V, dtype) if case["grad"] else None
        return s
    if T > 8:
        tokens[::97] = -100  # padding
    s["tokens"] = tokens.to(torch.int32)
    if op == "logprobs":
        s["logprob"], s["lse"] = torch.empty(T, **f32), torch.empty(T, **f32)
        s["entropy"] = torch.empty(T, **f32) if case["entropy"] else None
        s["top_index"] = torch.empty((T, k), **i32) if k else None
        s["top_logprob"] = torch.empty((T, k), **f32) if k else None
        return s
    # the way back: what the forward left, and the gradients that come in
    s["lse"], s["entropy"] = torch.empty(T, **f32), None
    if case["entropy"]:
        s["entropy"] = torch.empty(T, **f32)
    for a, b in _chunks(T, V, 1 << 27):
        z = s["logits"][a:b].double() / case["tau"]
        lse = torch.logsumexp(z, dim=1, keepdim=True)
        s["lse"][a:b] = lse[:, 0]
        if case["entropy"]:
            z -= lse
            s["entropy"][a:b] = -(torch.exp(z) * torch.where(z > -math.inf, z, 0.0)).sum(1)
    s["dlogprob"] = torch.randn(T, device="cuda", generator=g).div_(T)
    s["dentropy"] = torch.full((T,), -0.01 / T, device="cuda") if case["entropy"] else None
    s["dlogits"] = _space(T, V, dtype)
    return s


# ------------------------------------------------------------------ plain forms
def _softmax_parts(logits, tau):
    """z = logits / tau, the row's maximum, e^(z - max) and its sum."""
    z = logits.float() / tau
    top = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - top)
    return z, top, e, e.sum(dim=1, keepdim=True)


def _ranked(logits, k):
    """The k largest of each row, best first, ties to the lowest index: by a
    64-bit key, the value's order above the index's."""
    bits = (logits.float() + 0.0).view(torch.int32)
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF).long(), bits.long()) << 32
    key -= torch.arange(logits.shape[1], device="cuda")
    return (-key.topk(k, dim=1).values) & 0xFFFFFFFF


def _plain(s):
    case = s["case"]
    T, V, k, tau = case["T"], case["V"], case["k"], case["tau"]
    keep = torch.ones(T, device="cuda", dtype=torch.bool) if s["keep"] is None else s["keep"] != 0
    if case["op"] == "distill":
        return _plain_distill(s, keep)
    tokens = s["tokens"].long()
    inside = keep & (tokens >= 0) & (tokens < V)
    y = torch.where(inside, tokens, 0)[:, None]
    zero = torch.zeros((), device="cuda")
    if case["op"] == "logprobs":
        z, top, e, total = _softmax_parts(s["logits"], tau)
        less = top + torch.log(total)
        got = [torch.where(inside, (z.gather(1, y) - less)[:, 0], zero), torch.where(keep, less[:, 0], zero)]
        if case["entropy"]:
            d = torch.where(e > 0, z - top, zero)
            got.append(torch.where(keep, (torch.log(total) - (e * d).sum(1, keepdim=True) / total)[:, 0], zero))
            del d
        if k:
            index = _ranked(s["logits"], k)
            got.append(torch.where(keep[:, None], index, -1).to(torch.int32))
            got.append(torch.where(keep[:, None], z.gather(1, index) - less, zero))
        return got
    z = s["logits"].float() / tau
    logp = z - s["lse"][:, None]
    p = torch.exp(logp)
    g = torch.where(inside, s["dlogprob"], zero)
    d = -g[:, None] * p
    if case["entropy"]:
        d -= s["dentropy"][:, None] * p * (torch.where(p > 0, logp, zero) + s["entropy"][:, None])
    d.scatter_add_(1, y, g[:, None])
    return [torch.where(keep[:, None], d / tau, zero).to(s["dlogits"].dtype)]


def _plain_distill(s, keep):
    case = s["case"]
    T, V, tau = case["T"], case["V"], case["tau"]
    index = s["top_index"].long()
    present = ((index >= 0) & (index < V)).to(torch.int32).cumprod(1) > 0
    counted = keep & present[:, 0]
    n = counted.sum()
    zero = torch.zeros((), device="cuda")
    t = torch.where(present, s["top_logit"] / tau, -math.inf)
    t = torch.where(counted[:, None], t, zero)
    t = t - t.max(dim=1, keepdim=True).values
    w = torch.exp(t)
    q = w / w.sum(dim=1, keepdim=True)
    logq = t - torch.log(w.sum(dim=1, keepdim=True))
    z, top, e, total = _softmax_parts(s["logits"], tau)
    index = torch.where(present, index, 0)
    logp = z.gather(1, index) - top - torch.log(total)
    del z
    kl = torch.where(q > 0, q * (logq - logp), zero).sum(1)
    token = torch.where(counted, tau * tau * kl, zero)
    share = torch.where(n > 0, 1.0 / n, zero)
    got = [token, token.sum().reshape(1) * share, n.reshape(1).to(torch.int32)]
    if case["grad"]:
        e /= total
        e.scatter_add_(1, index, torch.where(present, -q, zero))
        e *= torch.where(counted, share * tau, zero)[:, None]
        got.append(e.to(s["dlogits"].dtype))
    return got


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import pmm_fc_layer_gb300 as fc
    case = s["case"]
    if case["op"] == "logprobs":
        fc.axonn_token_logprobs(s["logits"], tokens=s["tokens"], logprob=s["logprob"], entropy=s["entropy"],
                                lse=s["lse"], top_index=s["top_index"], top_logprob=s["top_logprob"],
                                keep=s["keep"], temperature=case["tau"])
        names = ["logprob", "lse"] + (["entropy"] if case["entropy"] else [])
        return [s[n] for n in names + (["top_index", "top_logprob"] if case["k"] else [])]
    if case["op"] == "logprobs_bwd":
        fc.axonn_token_logprobs_bwd(s["logits"], s["lse"], s["dlogits"], tokens=s["tokens"],
                                    dlogprob=s["dlogprob"], entropy=s["entropy"], dentropy=s["dentropy"],
                                    keep=s["keep"], temperature=case["tau"])
        return [s["dlogits"]]
    fc.axonn_distill(s["logits"], s["top_index"], s["top_logit"], s["token_loss"], s["loss"], s["kept"],
                     dlogits=s["dlogits"], keep=s["keep"], temperature=case["tau"])
    return [s["token_loss"], s["loss"], s["kept"]] + ([s["dlogits"]] if case["grad"] else [])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T, V, k, kept = case["T"], case["V"], case["k"], case["kept"]
    e = 4 if case["f32"] else 2
    read = T * kept * V * e  # masked rows need not be read
    mask = T if kept < 1 else 0
    if case["op"] == "logprobs":
        out = T * (4 + 4 + 4 + (4 if case["entropy"] else 0) + 8 * k)
        return {"bytes": read + out + mask, "flops": T * kept * V * (7 if case["entropy"] else 5)}
    if case["op"] == "logprobs_bwd":
        rows = T * (12 + (8 if case["entropy"] else 0))
        return {"bytes": read + T * V * e + rows + mask, "flops": T * kept * V * (9 if case["entropy"] else 5)}
    lists = T * kept * k * 8 * (0.5 if case["ragged"] else 1.0)
    out = T * V * e if case["grad"] else 0
    return {"bytes": read + out + lists + 4 * T + mask, "flops": T * kept * V * (9 if case["grad"] else 5)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    T, V, k, tau = case["T"], case["V"], case["k"], case["tau"]
    double = dict(device="cuda", dtype=torch.float64)
    rows = torch.arange(T, device="cuda") if s["keep"] is None else s["keep"].nonzero()[:, 0]
    if case["op"] == "distill":
        return _exact_distill(case, s, rows)
    tokens = s["tokens"].long()
    inside = (tokens >= 0) & (tokens < V)
    if case["op"] == "logprobs":
        logprob, lse, entropy = (torch.zeros(T, **double) for _ in range(3))
        index = torch.full((T, k), -1, device="cuda", dtype=torch.int32)
        value = torch.zeros((T, k), **double)
        for a, b in _chunks(rows.numel(), V, 1 << 27):
            r = rows[a:b]
            z = s["logits"][r].double() / tau
            logp = torch.log_softmax(z, dim=1)
            lse[r] = torch.logsumexp(z, dim=1)
            known = inside[r].nonzero()[:, 0]
            logprob[r[known]] = logp[known, tokens[r[known]]]
            if case["entropy"]:
                entropy[r] = torch.special.entr(logp.exp()).sum(1)
            if k:
                order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
                index[r], value[r] = order.to(torch.int32), logp.gather(1, order)
        got = [logprob, lse] + ([entropy] if case["entropy"] else [])
        return got + ([index, value] if k else [])
    d = torch.zeros((T, V), **double)
    for a, b in _chunks(rows.numel(), V, 1 << 27):
        r = rows[a:b]
        logp = s["logits"][r].double() / tau - s["lse"][r, None].double()
        p = logp.exp()
        g = torch.where(inside[r], s["dlogprob"][r].double(), 0.0)
        out = p * -g[:, None]
        if case["entropy"]:
            # p ln p is - entr(p), which is 0 at p = 0
            out -= s["dentropy"][r, None].double() * (p * s["entropy"][r, None].double() - torch.special.entr(p))
        at = torch.where(inside[r], tokens[r], 0)
        out[torch.arange(b - a, device="cuda"), at] += g
        d[r] = out / tau
    return [d]


def _exact_distill(case, s, rows):
    T, V, k, tau = case["T"], case["V"], case["k"], case["tau"]
    double = dict(device="cuda", dtype=torch.float64)
    # the length of each list: the place of its first index outside the vocabulary
    bad = (s["top_index"] < 0) | (s["top_index"] >= V)
    length = torch.where(bad.any(1), bad.to(torch.int8).argmax(1), k)
    rows = rows[length[rows] > 0]
    n = rows.numel()
    token = torch.zeros(T, **double)
    d = torch.zeros((T, V), **double) if case["grad"] else None
    for a, b in _chunks(n, V, 1 << 27):
        r = rows[a:b]
        here = torch.arange(k, device="cuda") < length[r, None]
        logq = torch.log_softmax(torch.where(here, s["top_logit"][r].double() / tau, -math.inf), dim=1)
        q = logq.exp()
        logp = torch.log_softmax(s["logits"][r].double() / tau, dim=1)
        at = torch.where(here, s["top_index"][r].long(), 0)
        token[r] = tau**2 * torch.where(here, q * (logq - logp.gather(1, at)), 0.0).sum(1)
        if case["grad"]:
            d[r] = logp.exp_().scatter_add_(1, at, -q) * (tau / n)
    return [token, token.sum().reshape(1) / max(n, 1), torch.tensor([n], dtype=torch.int32)] + (
        [d] if case["grad"] else [])
