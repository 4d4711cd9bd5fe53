"""The operators around a layer's products, as measured cases.

``run`` makes one pass through an operator: as a user calls it through
``pmm_fc_layer_gb300`` where ``own`` is true, else in plain torch operations
(32-bit arithmetic, one rounding at the end).  ``exact`` gives the same
outputs from the definition in 64 bits.  The operators:

fc_epi    Y = R + D(act(X W + b)), and Z = X W + b kept for the backward
dgrad_epi dZ = act'(Z) D(G W^T) + R, and db = column sums of act'(Z) D(G W^T)
act_bwd   dZ = act'(Z) D(dY), and db = its column sums
dropout   Y = R + D(X)
linear_ce cross entropy of the logits X W over a vocabulary: the loss of each
          token, their mean over the counted tokens, and its gradients

D(x) drops an element with probability p.  Its 16 random bits come from
Philox4x32-10 (Salmon et al., SC'11): key (seed low, seed high), counter
(col >> 3, row, offset low, offset high), 16-bit word col & 7 of the four
output words, lowest half first.  An element is dropped where they are below
thr = floor(65536 p + 1/2); the others are scaled by 65536 / (65536 - thr).
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _epi(op, name, T, K, N, act="none", bias="", p=0.0, res=False, pre=False, f32=False, wt=False):
    return {"name": name, "op": op, "T": T, "K": K, "N": N, "act": act, "bias": bias, "p": p,
            "res": res, "pre": pre, "f32": f32, "wt": wt}


def listed():
    return [
        # the two products of a GPT block's MLP (hidden 6144, 8192 tokens) in training: up with
        # GELU, its input kept for the backward; down with dropout, joined to the residual stream
        _epi("fc_epi", "up_gelu_train", 8192, 6144, 24576, "gelu_tanh", "bf16", pre=True),
        _epi("fc_epi", "down_dropout_residual_train", 8192, 24576, 6144, "none", "bf16", p=0.1, res=True),
        # the same MLP answering one token: the weights are read once and nothing else matters
        _epi("fc_epi", "up_gelu_token", 1, 6144, 24576, "gelu_tanh", "bf16"),
        # a ragged layer in PyTorch's Linear layout with an fp32 output
        _epi("fc_epi", "odd_silu_f32", 777, 1003, 2005, "silu", "f32", res=True, f32=True, wt=True),
        # the way back through the MLP: the data gradient of the down product, times GELU', with
        # the up layer's bias gradient
        _epi("dgrad_epi", "down_dgrad_gelu", 8192, 6144, 24576, "gelu_tanh", "f32"),
        # a small ragged step of the same, with dropout between the layers and a skip connection
        _epi("dgrad_epi", "odd_dgrad_relu_dropout", 300, 200, 1003, "relu", "f32", p=0.2, res=True),
        # a layer whose output gradient comes from elsewhere: elementwise, HBM-bound
        _epi("act_bwd", "act_bwd_gelu", 8192, 0, 24576, "gelu_tanh", "f32"),
        # dropout on the residual stream of the block, and of a few short sequences
        _epi("dropout", "dropout_residual", 8192, 0, 6144, p=0.1, res=True),
        _epi("dropout", "dropout_small_f32", 64, 0, 768, p=0.5, f32=True),
        # the loss over a 128256-token vocabulary: scoring a few tokens, and a training step
        {"name": "score_t16", "op": "linear_ce", "T": 16, "K": 6144, "V": 128256, "grad": False,
         "wt": False, "kept": 1.0},
        {"name": "loss_train_t4096", "op": "linear_ce", "T": 4096, "K": 6144, "V": 128256,
         "grad": True, "wt": False, "kept": 1.0},
        # embeddings tied to the head ([V x K]), an odd vocabulary, every second label left out
        # (the Goldfish rule's k = 2)
        {"name": "loss_tied_masked_odd", "op": "linear_ce", "T": 1003, "K": 768, "V": 50257,
         "grad": True, "wt": True, "kept": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fc_epi", "fc_epi", "dgrad_epi", "act_bwd", "dropout", "linear_ce", "linear_ce"])
    if op == "linear_ce":
        while True:
            T, K, V = _log(rng, 1, 8192), _log(rng, 64, 6144), _log(rng, 500, 128256)
            if T * K * V <= 4096 * 6144 * 128256:
                break
        return {"op": op, "T": T, "K": K, "V": V, "grad": rng.random() < 0.7,
                "wt": rng.random() < 0.5, "kept": rng.choice([1.0, 0.9, 0.5])}
    while True:
        T, K, N = _log(rng, 1, 8192), _log(rng, 32, 24576), _log(rng, 32, 24576)
        if T * K * N <= 8192 * 6144 * 24576:
            break
    c = _epi(op, "", T, K, N, rng.choice(ACTS), rng.choice(["", "bf16", "f32"]),
             rng.choice([0.0, 0.0, 0.1, 0.5]), rng.random() < 0.5, rng.random() < 0.5,
             rng.random() < 0.3, rng.random() < 0.5)
    del c["name"]
    if op == "dgrad_epi" or op == "act_bwd":
        c["bias"] = rng.choice(["", "f32"])
        c["pre"] = False
    if op == "act_bwd":
        c.update(K=0, res=False, wt=False)
    if op == "dropout":
        c.update(K=0, act="none", bias="", pre=False, wt=False, p=rng.choice([0.1, 0.3, 0.5]))
    return c


# ------------------------------------------------------------------ inputs
def _matrix(g, rows, cols, scale=1.0, dtype=BF16):
    """Rows with a leading dimension that is a multiple of 8, as the library wants it."""
    ld = (cols + 7) // 8 * 8
    full = torch.empty((rows, ld), device="cuda", dtype=dtype)
    step = max(1, (1 << 28) // ld)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        full[r:r + n] = torch.randn((n, ld), device="cuda", generator=g).mul_(scale)
    return full[:, :cols]


def _space(rows, cols, dtype=BF16):
    ld = (cols + 7) // 8 * 8
    return torch.empty((rows, ld), device="cuda", dtype=dtype)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T, K = case["op"], case["T"], case["K"]
    s = {"case": case}
    if op == "linear_ce":
        V = case["V"]
        s["X"] = _matrix(g, T, K)
        s["W"] = _matrix(g, V, K, 0.02) if case["wt"] else _matrix(g, K, V, 0.02)
        s["labels"] = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
        if T > 8:
            s["labels"][::97] = -100  # padding
        s["keep"] = None
        if case["kept"] < 1:
            s["keep"] = (torch.rand(T, device="cuda", generator=g) < case["kept"]).to(torch.uint8)
        s["token_loss"] = torch.empty(T, device="cuda")
        s["loss"] = torch.empty(1, device="cuda")
        s["kept"] = torch.empty(1, device="cuda", dtype=torch.int32)
        s["dX"] = _space(T, K) if case["grad"] else None
        s["dW"] = (_space(V, K) if case["wt"] else _space(K, V)) if case["grad"] else None
        s["ws"] = None  # the program's workspace, asked for at its first call
        return s
    N = case["N"]
    out = F32 if case["f32"] else BF16
    s["rng"] = torch.randint(-2**62, 2**62, (2,), device="cuda", generator=g)
    s["ws"] = None
    if op == "fc_epi":
        s["X"] = _matrix(g, T, K)
        s["W"] = _matrix(g, N, K, 0.02) if case["wt"] else _matrix(g, K, N, 0.02)
        s["bias"] = None
        if case["bias"]:
            s["bias"] = torch.randn(N, device="cuda", generator=g).mul_(0.1)
            s["bias"] = s["bias"].to(BF16) if case["bias"] == "bf16" else s["bias"]
        s["pre"] = _space(T, N) if case["pre"] else None
    elif op == "dgrad_epi":  # G [T x K] . W^T, W [N x K] as the forward of the next layer has it
        s["G"] = _matrix(g, T, K)
        s["W"] = _matrix(g, K, N, 0.02) if case["wt"] else _matrix(g, N, K, 0.02)
        s["Z"] = _matrix(g, T, N)
        s["db"] = torch.empty(N, device="cuda") if case["bias"] else None
    elif op == "act_bwd":
        s["dY"] = _matrix(g, T, N, dtype=out)
        s["Z"] = _matrix(g, T, N)
        s["db"] = torch.empty(N, device="cuda") if case["bias"] else None
        out = BF16
    else:
        s["X"] = _matrix(g, T, N, dtype=out)
    s["R"] = _matrix(g, T, N, dtype=out) if case["res"] else None
    s["Y"] = _space(T, N, out)
    return s


# ------------------------------------------------------------------ plain forms
def _mul_hi_lo(a, m):
    """The high and low words of a 32-bit product, in 64-bit integers that wrap."""
    prod = a * m
    return (prod >> 32) & 0xFFFFFFFF, prod & 0xFFFFFFFF


def _keep(rng, T, N, p):
    """The elements that D keeps, and their scale (None: keeps all)."""
    thr = int(math.floor(65536 * p + 0.5))
    if thr == 0:
        return None, 1.0
    n8 = (N + 7) // 8
    seed, offset = rng[0], rng[1]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    c0 = torch.arange(n8, device="cuda").expand(T, n8)
    c1 = torch.arange(T, device="cuda")[:, None].expand(T, n8)
    c2 = (offset & 0xFFFFFFFF).expand(T, n8)
    c3 = ((offset >> 32) & 0xFFFFFFFF).expand(T, n8)
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16,
                         c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], dim=2).reshape(T, 8 * n8)
    return words[:, :N] >= thr, (65536 / (65536 - thr) if thr < 65536 else 0.0)


def _drop(x, rng, p):
    keep, scale = _keep(rng, x.shape[0], x.shape[1], p)
    return x if keep is None else torch.where(keep, x * scale, torch.zeros_like(x))


_RT2, _RT2PI, _T0, _T1 = math.sqrt(0.5), 1 / math.sqrt(2 * math.pi), math.sqrt(2 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * _RT2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_T0 * (z + _T1 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * _RT2)) + z * _RT2PI * torch.exp(-0.5 * z * z)
    if act == "gelu_tanh":
        t = torch.tanh(_T0 * (z + _T1 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _T0 * (1 + 3 * _T1 * z * z)
    if act == "silu":
        e = 1 / (1 + torch.exp(-z))
        return e * (1 + z * (1 - e))
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    op, act, p = case["op"], case.get("act"), case.get("p")
    if op == "linear_ce":
        return _plain_ce(s)
    out = s["Y"].dtype
    if op == "fc_epi":
        W = s["W"].float()
        z = s["X"].float() @ (W.t() if case["wt"] else W)
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _drop(_act(z, act), s["rng"], p)
        y = y if s["R"] is None else y + s["R"].float()
        return [y.to(out)] + ([z.to(BF16)] if case["pre"] else [])
    if op == "dropout":
        y = _drop(s["X"].float(), s["rng"], p)
        return [(y if s["R"] is None else y + s["R"].float()).to(out)]
    if op == "dgrad_epi":
        W = s["W"].float()
        d = s["G"].float() @ (W if case["wt"] else W.t())
    else:
        d = s["dY"].float()
    d = _drop(d, s["rng"], p) * _dact(s["Z"].float(), act)
    y = d if s["R"] is None else d + s["R"].float()
    return [y.to(out)] + ([d.sum(0)] if case["bias"] else [])


def _plain_ce(s):
    case = s["case"]
    T, V = case["T"], case["V"]
    X, W = s["X"].float(), s["W"].float()
    W = W.t() if case["wt"] else W
    labels = s["labels"].long()
    counted = (labels >= 0) & (labels < V)
    if s["keep"] is not None:
        counted = counted & (s["keep"] != 0)
    y = torch.where(counted, labels, torch.zeros_like(labels))
    n = counted.sum()
    z = X @ W
    top = z.max(dim=1, keepdim=True).values
    zy = z.gather(1, y[:, None])
    e = torch.exp(z - top)
    del z
    total = e.sum(dim=1, keepdim=True)
    zero = torch.zeros(1, device="cuda")
    token = torch.where(counted, (top + torch.log(total) - zy)[:, 0], zero)
    share = torch.where(n > 0, 1.0 / n, zero)
    got = [token, token.sum().reshape(1) * share, n.reshape(1).to(torch.int32)]
    if case["grad"]:
        e /= total
        e.scatter_add_(1, y[:, None], torch.full((T, 1), -1.0, device="cuda"))
        e *= torch.where(counted, share, zero)[:, None]
        got.append((e @ W.t()).to(BF16))
        got.append((e.t() @ X if case["wt"] else X.t() @ e).to(BF16))
    return got


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import pmm_fc_layer_gb300 as fc
    case = s["case"]
    op, T, K = case["op"], case["T"], case["K"]
    if op == "linear_ce":
        flags = fc.B_T if case["wt"] else 0
        if s["ws"] is None:
            nbytes = fc.axonn_linear_ce_workspace_size(T, K, case["V"], flags, grad=case["grad"])
            s["ws"] = torch.empty(max(nbytes, 16), device="cuda", dtype=torch.uint8)
        fc.axonn_linear_ce(s["X"], s["W"], s["labels"], s["token_loss"], s["loss"], s["kept"],
                           ws=s["ws"], keep=s["keep"], dX=s["dX"], dW=s["dW"], flags=flags)
        got = [s["token_loss"], s["loss"], s["kept"]]
        return got + ([s["dX"], s["dW"]] if case["grad"] else [])
    N, p, act = case["N"], case["p"], case["act"]
    rng = s["rng"] if p > 0 else None
    if op == "dropout":
        fc.axonn_dropout(s["X"], s["Y"], p, rng, residual=s["R"])
        return [s["Y"]]
    if op == "fc_epi":
        flags = (fc.B_T if case["wt"] else 0) | (fc.OUT_F32 if case["f32"] else 0)
        fc.axonn_fc_fwd_epi(s["X"], s["W"], s["Y"], fc.Shape(T, K, N), flags, bias=s["bias"], act=act,
                            pre=s["pre"], residual=s["R"], p=p, rng=rng)
        return [s["Y"]] + ([s["pre"]] if case["pre"] else [])
    if s["ws"] is None:
        nbytes = fc.axonn_epi_workspace_size(T, N)
        s["ws"] = torch.empty(max(nbytes, 16), device="cuda", dtype=torch.uint8)
    ws = s["ws"] if case["bias"] else None
    if op == "dgrad_epi":
        # dX [T x N] of the product whose forward is [T x N] . W[N x K]
        flags = (fc.B_T if case["wt"] else 0) | (fc.OUT_F32 if case["f32"] else 0)
        fc.axonn_fc_dgrad_epi(s["G"], s["W"], s["Y"], fc.Shape(T, N, K), flags, pre=s["Z"], act=act,
                              residual=s["R"], dbias=s["db"], p=p, rng=rng, ws=ws)
    else:
        fc.axonn_epi_bwd(s["dY"], s["Y"], pre=s["Z"], act=act, dbias=s["db"], p=p, rng=rng, ws=ws)
    return [s["Y"]] + ([s["db"]] if case["bias"] else [])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, T, K = case["op"], case["T"], case["K"]
    if op == "linear_ce":
        V = case["V"]
        n = T * case["kept"]  # rows whose label counts; the others need no logits
        b = 2 * n * K + 2 * K * V + 5 * T + 4 * T
        if case["grad"]:
            return {"bytes": b + 2 * T * K + 2 * K * V, "flops": 6 * n * K * V}
        return {"bytes": b, "flops": 2 * n * K * V}
    N, e = case["N"], 4 if case["f32"] else 2
    b = T * N * e * (2 if case["res"] else 1)  # output and residual
    if op == "dropout":
        return {"bytes": b + T * N * e, "flops": T * N}
    if op == "act_bwd":
        z = 2 if case["act"] != "none" else 0
        return {"bytes": T * N * (e + z + 2) + (4 * N if case["bias"] else 0), "flops": 10 * T * N}
    b += 2 * T * K + 2 * K * N
    if op == "fc_epi":
        b += (2 * T * N if case["pre"] else 0) + {"": 0, "bf16": 2 * N, "f32": 4 * N}[case["bias"]]
    else:
        b += (2 * T * N if case["act"] != "none" else 0) + (4 * N if case["bias"] else 0)
    return {"bytes": b, "flops": 2 * T * K * N}


# ------------------------------------------------------------------ 64 bits
def _exact_drop(x, rng, p):
    thr = math.floor(65536 * p + 0.5)
    if thr == 0:
        return x
    T, N = x.shape
    n8 = -(-N // 8)
    seed, offset = (int(v) % 2**64 for v in rng.tolist())
    low = np.uint64(0xFFFFFFFF)
    c = [np.broadcast_to(np.arange(n8, dtype=np.uint64), (T, n8)),
         np.broadcast_to(np.arange(T, dtype=np.uint64)[:, None], (T, n8)),
         np.full((T, n8), offset % 2**32, np.uint64), np.full((T, n8), offset >> 32, np.uint64)]
    key = [seed % 2**32, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(key[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    bits = np.stack(c, axis=2).astype("<u4").view("<u2").reshape(T, 8 * n8)[:, :N]
    m = torch.from_numpy(bits >= thr).to(x.device)
    return torch.where(m, x * (65536.0 / (65536 - thr) if thr < 65536 else 0.0), torch.zeros_like(x))


def _exact_act(z, act):
    import torch.nn.functional as F
    return {"none": lambda v: v * 1.0, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[act](z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear_ce":
        return _exact_ce(case, s)
    if case["p"] > 0 and case["T"] * case["N"] > 6e7:  # the generator in 64 bits on the host
        return None
    if op == "fc_epi":
        W = s["W"].double()
        z = torch.matmul(s["X"].double(), W.mT if case["wt"] else W)
        z = z if s["bias"] is None else z + s["bias"].double()
        y = _exact_drop(_exact_act(z, case["act"]), s["rng"], case["p"])
        return [y if s["R"] is None else y + s["R"].double()] + ([z] if case["pre"] else [])
    if op == "dropout":
        y = _exact_drop(s["X"].double(), s["rng"], case["p"])
        return [y if s["R"] is None else y + s["R"].double()]
    if op == "dgrad_epi":
        W = s["W"].double()
        d = torch.matmul(s["G"].double(), W if case["wt"] else W.mT)
    else:
        d = s["dY"].double()
    d = _exact_drop(d, s["rng"], case["p"])
    z = s["Z"].double().requires_grad_(True)
    d = torch.autograd.grad(_exact_act(z, case["act"]), z, d)[0]
    return [d if s["R"] is None else d + s["R"].double()] + ([d.sum(0)] if case["bias"] else [])


def _exact_ce(case, s):
    T, K, V = case["T"], case["K"], case["V"]
    X, W = s["X"].double(), s["W"].double()
    W = W.mT if case["wt"] else W
    ok = (s["labels"] >= 0) & (s["labels"] < V)
    if s["keep"] is not None:
        ok &= s["keep"] != 0
    rows = ok.nonzero()[:, 0]
    n = rows.numel()
    y = s["labels"][rows].long()
    z = X[rows] @ W
    logp = torch.log_softmax(z, dim=1)
    del z
    token = torch.zeros(T, device="cuda", dtype=torch.float64)
    token[rows] = -logp[torch.arange(n, device="cuda"), y]
    got = [token, (token.sum() / max(n, 1)).reshape(1), torch.tensor([n], dtype=torch.int32)]
    if case["grad"]:
        if 6 * n * K * V > 1.2e13:  # more than the 64-bit rate gives in a few seconds
            return got + [None, None]
        P = logp.exp_()
        P[torch.arange(n, device="cuda"), y] -= 1
        P /= max(n, 1)
        dX = torch.zeros((T, K), device="cuda", dtype=torch.float64)
        dX[rows] = P @ W.mT
        got += [dX, P.mT @ X[rows] if case["wt"] else X[rows].mT @ P]
    return got
