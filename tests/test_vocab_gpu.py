"""The operators over rows of vocabulary logits against their 64-bit forms.

Bounds (derived).  D_v = (m - x_v) / tau is a logit's distance from the row's
maximum.  The kernel's exponent d = (x - m) c has three relative roundings (the
difference, c = log2(e) / tau with two of its own, the product), so 2^d is off
by D 2^-22 of itself and by 2^-22 for the function unit.  S is a sum of such
terms: off by E = 2^-22 (1 + sum p D) of itself and by 2^-24 for each of at most
V / 2048 + 48 additions on the way of a term (a thread's own, the warp's, the
block's), and ln S by that and 2^-22 |ln S| for the logarithm and its factor.
  ln p    E + 2^-21 (D + ln S), the exponent's roundings and the last ones
  lse     E + 2^-22 (|lse| + |m / tau|)
  H       ln S - A / S: E (1 + sum p D), each term of A by D (D + 2) 2^-22 of p,
          2^-22 (ln S + sum p D)
  forward's p in the distillation: E + (D + 2) 2^-22 of itself
  backward's p: lse is given, so |x / tau| 2^-23 + (|ln p| + 1) 2^-22 of itself
An output in fewer bits is rounded once: half a step, 2^-8 (bf16) or 2^-24 of it.
Exponentials below 2^-126 are 0.
"""
import numpy as np
import pytest

from oracle import vocab as vo

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0**-8, "f32": 2.0**-24}
TINY = 1e-36


def kind_of(kind):
    import torch
    return torch.bfloat16 if kind == "bf16" else torch.float32


def stored(x, kind):
    """x as the type holds it, in 64 bits."""
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to(kind_of(kind)).to(torch.float64).numpy()


def rows_on_gpu(x, kind, pad=8, fill=float("nan")):
    """[T x V] inside rows of more columns, whose others are `fill`."""
    import torch
    T, V = x.shape
    full = torch.full((T, (V + 7) // 8 * 8 + pad), fill, dtype=kind_of(kind), device="cuda")
    full[:, :V] = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(kind_of(kind))
    return full[:, :V]


def gpu(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(a):
    import torch
    return gpu(np.asarray(a)).to(torch.int32)


def f32(a):
    return gpu(np.asarray(a, np.float32))


def host(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def padding_untouched(t, fill=float("nan")):
    import torch
    rest = t._base[:, t.shape[1]:].float()
    return bool((torch.isnan(rest) if fill != fill else rest == fill).all())


def numbers(x, tau):
    """D, p, ln S, sum p D and E of every row."""
    V = x.shape[1]
    with np.errstate(invalid="ignore", over="ignore"):
        D = (x.max(axis=1, keepdims=True) - x) / tau
    D = np.where(np.isnan(D), 0.0, D)
    p = np.exp(-D)
    S = p.sum(axis=1, keepdims=True)
    p = p / S
    pD = np.where(p > 0, p * np.where(p > 0, D, 0), 0).sum(axis=1)
    E = 2.0**-22 * (1 + pD) + 2.0**-24 * (V / 2048 + 48) + 2.0**-22 * np.log(S[:, 0])
    return D, p, np.log(S[:, 0]), pD, E


def close(got, want, tol, what):
    with np.errstate(over="ignore"):  # beyond fp32 it is an infinity
        want = np.where(np.abs(want) > np.finfo(np.float32).max, np.float64(np.float32(want)), want)
    got, want, tol = np.broadcast_arrays(got, want, tol)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


# ------------------------------------------------------------------ logprobs
def run_logprobs(fc, x, kind, tokens, keep=None, tau=1.0, k=0, entropy=True):
    import torch
    T = x.shape[0]
    X = rows_on_gpu(x, kind)
    o = {n: torch.full((T,), 7.0, device="cuda") for n in ("logprob", "lse") + (("entropy",) if entropy else ())}
    if k:
        o["top_index"] = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
        o["top_logprob"] = torch.full((T, k), 7.0, device="cuda")
    fc.axonn_token_logprobs(X, tokens=i32(tokens), keep=None if keep is None else gpu(keep.astype(np.uint8)),
                            temperature=tau, **o)
    fc.axonn_sync_status()
    return {n: host(t) for n, t in o.items()}


def check_logprobs(got, x, tokens, keep=None, tau=1.0, k=0):
    T, V = x.shape
    tau = float(np.float32(tau))
    want = vo.token_logprobs(x, tokens, keep, tau, k)
    D, p, lnS, pD, E = numbers(x, tau)
    y = np.where((tokens >= 0) & (tokens < V), tokens, 0)
    close(got["logprob"], want["logprob"], E + 2.0**-21 * (D[np.arange(T), y] + lnS), "logprob")
    with np.errstate(invalid="ignore"):
        top = np.abs(x.max(axis=1)) / tau
    close(got["lse"], want["lse"], E + 2.0**-22 * (np.abs(want["lse"]) + top), "lse")
    if "entropy" in got:
        pDD = np.where(p > 0, p * np.where(p > 0, D * (D + 2), 0), 0).sum(axis=1)
        close(got["entropy"], want["entropy"], E * (1 + pD) + 2.0**-22 * (pDD + lnS + pD), "entropy")
    if k:
        assert np.array_equal(got["top_index"], want["top_index"])
        at = np.maximum(want["top_index"], 0)
        tol = E[:, None] + 2.0**-21 * (np.take_along_axis(D, at, 1) + lnS[:, None])
        close(got["top_logprob"], want["top_logprob"], tol, "top_logprob")


def logits_of(T, V, kind, seed=1, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, V)) * spread
    tokens = rng.integers(0, V, size=T)
    x[np.arange(T), tokens] += rng.uniform(0, 12, size=T)
    return stored(x, kind), tokens, rng


SIZES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 130), (4, 1003), (3, 4096), (2, 4099), (3, 16384), (2, 33333),
         (170, 600), (1, 131075), (2, 200001)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_logprobs_against_64_bits(cuda_lib, size, kind):
    T, V = size
    x, tokens, _ = logits_of(T, V, kind)
    for k in sorted({0, 1, min(V, 5), min(V, 20), min(V, 128)}):
        check_logprobs(run_logprobs(cuda_lib, x, kind, tokens, k=k), x, tokens, k=k)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [0.5, 0.7, 3.0])
def test_logprobs_temperature_mask_and_padding(cuda_lib, kind, tau):
    x, tokens, rng = logits_of(40, 2007, kind, seed=5)
    tokens[::7] = -100
    tokens[3], tokens[5] = 2007, 2006
    keep = (rng.random(40) < 0.6).astype(np.uint8)
    x[keep == 0] = np.nan  # never read
    clean = np.where(np.isnan(x), 0.0, x)
    for entropy in (False, True):
        got = run_logprobs(cuda_lib, x, kind, tokens, keep, tau, 9, entropy)
        check_logprobs(got, clean, tokens, keep, tau, 9)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,ks", [(650, 700, (1, 64, 65)), (700, 9001, (3, 64)), (2500, 300, (2, 10, 11, 24, 25)),
                                    (3700, 2100, (1, 10)), (610, 20003, (20,))])
def test_logprobs_many_rows(cuda_lib, T, V, ks, kind):
    """Blocks of every size: few threads for many short rows."""
    x, tokens, _ = logits_of(min(T, 97), V, kind, seed=16)
    x[::5] = np.round(x[::5])  # ties
    pick = np.arange(T) % len(x)
    for k in ks:
        for entropy in (False, True):
            got = run_logprobs(cuda_lib, x[pick], kind, tokens[pick], k=k, entropy=entropy)
            check_logprobs({n: v[:len(x)] for n, v in got.items()}, x, tokens, k=k)
            for n, v in got.items():
                assert np.array_equal(v, v[:len(x)][pick]), n


def special_rows(V, kind):
    """Rows that are hard on a maximum, a sum or an order."""
    rng = np.random.default_rng(9)
    low = -3.3895313892515355e38 if kind == "bf16" else float(np.finfo(np.float32).min)
    rows = {
        "constant": np.full(V, 1.5),
        "all lowest": np.full(V, low),
        "lowest but one": np.where(np.arange(V) == V // 2, -4.0, low),
        "huge": np.where(np.arange(V) % 5 == 0, -low / 2, low),
        "empty": np.full(V, -np.inf),
        "one left": np.where(np.arange(V) == V - 1, 3.0, -np.inf),
        "three left": np.where(np.isin(np.arange(V), [0, V // 3, V - 2]), 2.0, -np.inf),
        "zeros of both signs": np.where(np.arange(V) % 2 == 0, -0.0, 0.0),
        "ascending": np.arange(V) / V * 8,
        "descending": -np.arange(V) / V * 8,
        "few values": rng.integers(-2, 3, size=V).astype(float),
        "far away": rng.normal(size=V) + 500,
        "best in one column of threads": np.where(np.arange(V) % 4096 < 8, 5.0, 0.0) + rng.normal(size=V),
        "best behind one another": np.where(np.arange(V) // 512 == 1, 9.0, 0.0) + np.arange(V) % 64 / 64,
        "tiny": rng.normal(size=V) * 1e-39,
        "a NaN": np.where(np.arange(V) == V // 4, np.nan, rng.normal(size=V)),
        "NaN of both signs": np.where(np.arange(V) % 1000 == 3, -np.nan, np.where(np.arange(V) % 999 == 1, np.nan, 1.0)),
        "all NaN": np.full(V, np.nan),
        "an infinity": np.where(np.arange(V) == 5 % V, np.inf, rng.normal(size=V)),
        "infinities and NaN": np.where(np.arange(V) % 7 == 5, np.inf, np.where(np.arange(V) % 7 == 6, np.nan, -np.inf)),
    }
    return list(rows), stored(np.stack(list(rows.values())), kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [8, 1003, 8200, 70001])
@pytest.mark.parametrize("k", [1, 8, 100])
def test_logprobs_special_rows(cuda_lib, V, kind, k):
    names, x = special_rows(V, kind)
    k = min(k, V)
    tokens = np.full(len(names), V // 2)
    got = run_logprobs(cuda_lib, x, kind, tokens, k=k)
    want = vo.token_logprobs(x, tokens, None, 1.0, k)
    with np.errstate(invalid="ignore"):
        D, p, lnS, pD, E = numbers(np.where(np.isfinite(x), x, -np.inf), 1.0)
    for t, name in enumerate(names):
        assert np.array_equal(got["top_index"][t], want["top_index"][t]), (name, got["top_index"][t][:9])
        if not np.isfinite(want["lse"][t]):
            for n in ("logprob", "lse", "entropy", "top_logprob"):
                close(got[n][t], want[n][t], 0.0, (name, n))
    fine = np.isfinite(want["lse"])
    check_logprobs({n: v[fine] for n, v in got.items()}, x[fine], tokens[fine], None, 1.0, k)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 2000])
def test_lists_of_rows_with_what_is_large_in_a_few_threads(cuda_lib, T, kind):
    """More logits reach the bound that the threads' best give than a block
    holds: one vector of eight in four, at a stride that gives them to 60
    threads."""
    V, k = 65541, 100
    rng = np.random.default_rng(15)
    x = rng.normal(size=(3, V)) + np.where(np.arange(V) // 8 % 256 < 60, 9.0, 0.0)
    x = stored(np.repeat(x, T // 3 + 1, axis=0)[:T], kind)
    got = run_logprobs(cuda_lib, x, kind, np.zeros(T, int), k=k)
    pick = np.unique([0, 1, 2, T // 2, T - 1])
    check_logprobs({n: v[pick] for n, v in got.items()}, x[pick], np.zeros(len(pick), int), k=k)


def test_logprobs_each_output_alone(cuda_lib):
    import torch
    x, tokens, _ = logits_of(6, 3001, "bf16", seed=3)
    X = rows_on_gpu(x, "bf16")
    full = run_logprobs(cuda_lib, x, "bf16", tokens, k=4)
    for name, shape, dtype in (("entropy", (6,), torch.float32), ("lse", (6,), torch.float32),
                               ("top_index", (6, 4), torch.int32), ("top_logprob", (6, 4), torch.float32)):
        o = torch.zeros(shape, dtype=dtype, device="cuda")
        cuda_lib.axonn_token_logprobs(X, **{name: o})
        assert np.array_equal(host(o), full[name]), name
    o = torch.zeros(6, device="cuda")
    cuda_lib.axonn_token_logprobs(X, tokens=i32(tokens), logprob=o)
    assert np.array_equal(host(o), full["logprob"])


def test_lists_with_a_row_stride(cuda_lib):
    import torch
    x, tokens, _ = logits_of(5, 700, "f32", seed=4)
    X = rows_on_gpu(x, "f32")
    index = torch.full((5, 13), -9, dtype=torch.int32, device="cuda")
    value = torch.full((5, 13), 7.0, device="cuda")
    cuda_lib.axonn_token_logprobs(X, top_index=index[:, 2:9], top_logprob=value[:, 2:9])
    want = vo.token_logprobs(x, None, None, 1.0, 7)
    assert np.array_equal(host(index)[:, 2:9], want["top_index"])
    assert (host(index)[:, :2] == -9).all() and (host(index)[:, 9:] == -9).all()
    assert (host(value)[:, :2] == 7).all() and (host(value)[:, 9:] == 7).all()
    with pytest.raises(ValueError):
        cuda_lib.axonn_token_logprobs(X, top_index=index[:, :7], top_logprob=value[:, :7].contiguous())


# ------------------------------------------------------------------ logprobs, backward
def run_backward(fc, x, kind, lse, tokens=None, g=None, H=None, h=None, keep=None, tau=1.0, in_place=False):
    X = rows_on_gpu(x, kind)
    out = X if in_place else rows_on_gpu(np.full(x.shape, 7.0), kind)
    fc.axonn_token_logprobs_bwd(X, f32(lse), out, tokens=None if tokens is None else i32(tokens),
                                dlogprob=None if g is None else f32(g), entropy=None if H is None else f32(H),
                                dentropy=None if h is None else f32(h),
                                keep=None if keep is None else gpu(keep.astype(np.uint8)), temperature=tau)
    fc.axonn_sync_status()
    assert padding_untouched(out)
    return host(out)


def check_backward(got, x, kind, lse, tokens=None, g=None, H=None, h=None, keep=None, tau=1.0):
    T, V = x.shape
    tau = float(np.float32(tau))
    want = vo.token_logprobs_bwd(x, lse, tokens, g, H, h, keep, tau)
    lse = np.asarray(lse, np.float64)
    with np.errstate(invalid="ignore"):
        lp = x / tau - lse[:, None]
        p = np.exp(lp)
    lp = np.where(p > 0, lp, 0.0)
    z = np.where(p > 0, np.abs(x) / tau, 0.0)
    ep = z * 2.0**-23 + (np.abs(lp) + 1) * 2.0**-22
    G = np.zeros((T, 1)) if g is None else np.abs(np.float64(g))[:, None]
    hh = np.zeros((T, 1)) if h is None else np.abs(np.float64(h))[:, None]
    HH = np.zeros((T, 1)) if H is None else np.abs(np.float64(H))[:, None]
    w = G + hh * (np.abs(lp) + HH)
    tol = p * (w * (ep + 2.0**-21) + hh * z * 2.0**-23) + G * 2.0**-22 * (p + (np.arange(V) == (
        np.full(T, -1) if tokens is None else tokens)[:, None]))
    close(got, want, tol / tau + HALF[kind] * np.abs(want) + TINY, "dlogits")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_backward_against_64_bits(cuda_lib, size, kind, in_place):
    T, V = size
    x, tokens, rng = logits_of(T, V, kind, seed=11)
    tau = 0.8
    f = vo.token_logprobs(x, tokens, None, float(np.float32(tau)))
    lse, H = f["lse"].astype(np.float32), f["entropy"].astype(np.float32)
    g, h = rng.normal(size=T).astype(np.float32), rng.normal(size=T).astype(np.float32)
    for kw in (dict(tokens=tokens, g=g), dict(tokens=tokens, g=g, H=H, h=h), dict(H=H, h=h)):
        got = run_backward(cuda_lib, x, kind, lse, tau=tau, in_place=in_place, **kw)
        check_backward(got, x, kind, lse, tau=tau, **kw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_backward_masks_and_masked_logits(cuda_lib, kind):
    x, tokens, rng = logits_of(30, 1500, kind, seed=12)
    x[rng.random(x.shape) < 0.7] = -np.inf
    x[np.arange(30), tokens] = 1.0
    x[4] = -np.inf                         # an empty row: no gradient
    low = stored(np.array([-3.38e38]), kind)[0]
    x[5, 1:] = low                         # a mask of the type's lowest value
    x[5, 0] = 1.0
    f = vo.token_logprobs(x, tokens)
    lse, H = f["lse"].astype(np.float32), f["entropy"].astype(np.float32)
    g, h = rng.normal(size=30).astype(np.float32), rng.normal(size=30).astype(np.float32)
    tokens[::6] = -100
    tokens[7] = 1500
    keep = (rng.random(30) < 0.7).astype(np.uint8)
    keep[4:8] = 1
    g[9] = h[9] = 0
    x[9] = np.nan                          # no gradient comes in: zeros
    x[keep == 0] = np.nan
    got = run_backward(cuda_lib, x, kind, lse, tokens, g, H, h, keep)
    assert (got[4] == 0).all() and (got[9] == 0).all() and (got[keep == 0] == 0).all()
    check_backward(got, np.where(np.isnan(x), 0.0, x), kind, lse, tokens, g, H, h, keep)


def test_backward_of_a_row_that_is_not_a_number(cuda_lib):
    x, tokens, _ = logits_of(2, 100, "f32")
    got = run_backward(cuda_lib, x, "f32", np.array([np.nan, 3.0]), tokens, np.ones(2))
    assert np.isnan(got[0]).all() and np.isfinite(got[1]).all()


def test_backward_against_differences(cuda_lib):
    """The gradient of g . logprob + h . entropy, by differences of the kernel's
    own forward along random directions: with step s, s^2 f'''/6 and the
    forward's errors over s, both below 2e-3 of the sums' size here."""
    T, V, tau, s = 4, 300, 0.9, 2e-2
    x, tokens, rng = logits_of(T, V, "f32", seed=13, spread=1.0)
    g, h = rng.normal(size=T), rng.normal(size=T)
    f = run_logprobs(cuda_lib, x, "f32", tokens, tau=tau)
    d = run_backward(cuda_lib, x, "f32", f["lse"], tokens, g, f["entropy"], h, tau=tau)

    def value(v):
        r = run_logprobs(cuda_lib, stored(v, "f32"), "f32", tokens, tau=tau)
        return g @ r["logprob"] + h @ r["entropy"]
    for _ in range(6):
        u = rng.normal(size=x.shape)
        u /= np.linalg.norm(u)
        assert abs((value(x + s * u) - value(x - s * u)) / (2 * s) - (d * u).sum()) < 2e-3


# ------------------------------------------------------------------ distillation
def run_distill(fc, x, kind, at, t, keep=None, tau=1.0, scale=1.0, grad=True, in_place=False):
    import torch
    T = x.shape[0]
    X = rows_on_gpu(x, kind)
    out = None if not grad else X if in_place else rows_on_gpu(np.full(x.shape, 7.0), kind)
    token = torch.full((T,), 7.0, device="cuda")
    loss, kept = torch.full((1,), 7.0, device="cuda"), torch.full((1,), -7, dtype=torch.int32, device="cuda")
    fc.axonn_distill(X, i32(at), f32(t), token, loss, kept, dlogits=out,
                     keep=None if keep is None else gpu(keep.astype(np.uint8)), temperature=tau, grad_scale=scale)
    fc.axonn_sync_status()
    got = {"token_loss": host(token), "loss": host(loss)[0], "kept": int(kept.item())}
    if grad:
        assert padding_untouched(out)
        got["dlogits"] = host(out)
    return got


def check_distill(got, x, kind, at, t, keep=None, tau=1.0, scale=1.0):
    T, V = x.shape
    tau = float(np.float32(tau))
    want = vo.distill(x, at, t, keep, tau, scale)
    n = max(want["n"], 1)
    assert got["kept"] == want["n"]
    D, p, lnS, pD, E = numbers(x, tau)
    tol = np.zeros(T)
    eq = np.zeros((T, V))
    for r in np.nonzero(want["counted"])[0]:
        inside = (at[r] >= 0) & (at[r] < V)
        L = len(inside) if inside.all() else int(np.argmin(inside))
        a = at[r, :L]
        Dt, q, lnW, qD, Et = (v[0] for v in numbers(np.float64(t[r:r + 1, :L]), tau))
        q = np.where(np.isfinite(q), q, 0.0)  # a list of -inf alone
        Dt, Ds = np.where(q > 0, Dt, 0), np.where(q > 0, D[r, a], 0)
        relq = Et + (Dt + 2) * 2.0**-22
        each = Et + E[r] + 2.0**-21 * (Dt + Ds + lnW + lnS[r])
        size = np.abs(-Dt - lnW + Ds + lnS[r])
        tol[r] = (q * (each + size * (relq + 2.0**-24 * (L / 32 + 8)))).sum() * tau**2
        np.add.at(eq[r], a, q * relq + q * 2.0**-24 * L)
    close(got["token_loss"], want["token_loss"], tol + 2.0**-22 * np.abs(want["token_loss"]), "token_loss")
    mean_tol = (tol.sum() + np.abs(want["token_loss"]).sum() * (T / 512 + 32) * 2.0**-24) / n
    close(got["loss"], want["loss"], mean_tol + 2.0**-22 * abs(want["loss"]), "loss")
    if "dlogits" in got:
        c = want["counted"][:, None]
        D0 = np.where(p > 0, D, 0.0)
        near = p * (E[:, None] + (D0 + 2) * 2.0**-22 + 2.0**-22)
        q_size = np.abs(want["dlogits"] / (scale * tau / n) - p)
        bound = (near + eq + 2.0**-22 * q_size) * abs(scale) * tau / n
        close(got["dlogits"], want["dlogits"], np.where(c, bound + HALF[kind] * np.abs(want["dlogits"]) + TINY, 0.0),
              "dlogits")


def lists_of(x, k, rng, noise=0.5):
    """A teacher near the student: its k best."""
    teacher = np.where(np.isfinite(x), x, -5.0) + noise * rng.normal(size=x.shape)
    at = np.argsort(-teacher, axis=1, kind="stable")[:, :k]
    return at, np.take_along_axis(teacher, at, 1).astype(np.float32)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_distill_against_64_bits(cuda_lib, size, kind):
    T, V = size
    x, _, rng = logits_of(T, V, kind, seed=21)
    for k, tau in ((1, 1.0), (min(V, 9), 2.0), (min(V, 64), 0.7), (min(V, 600), 1.0)):
        at, t = lists_of(x, k, rng)
        check_distill(run_distill(cuda_lib, x, kind, at, t, tau=tau), x, kind, at, t, tau=tau)
    check_distill(run_distill(cuda_lib, x, kind, at, t, grad=False), x, kind, at, t)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_distill_lists_and_masks(cuda_lib, kind, in_place):
    V = 1100
    x, _, rng = logits_of(40, V, kind, seed=22)
    at, t = lists_of(x, 12, rng)
    length = rng.integers(0, 13, size=40)
    length[0], length[1], length[2] = 0, 1, 12
    at[np.arange(12) >= length[:, None]] = -1
    at[3, 2] = V                           # ends the list
    at[4, :] = at[4, 0]                    # the same index twelve times
    at[5, 6:] = at[5, :6]
    t[6, 1:] = -np.inf
    t[7, :] = -np.inf                      # a list that teaches nothing
    length[4:8] = 12
    at[6], at[7] = lists_of(x[6:8], 12, rng)[0]
    x[8] = -np.inf                         # a student without a word left
    at[8], t[8] = np.arange(12) * 50, rng.normal(size=12)
    x[10, at[10, 0]] = -np.inf             # p = 0 where q > 0
    if at[10, 0] < 0:
        at[10] = np.arange(12)
        x[10, 0] = -np.inf
    keep = (rng.random(40) < 0.7).astype(np.uint8)
    keep[:11] = 1
    skipped = (keep == 0) | (at[:, 0] < 0)
    x[skipped] = np.nan                    # never read
    got = run_distill(cuda_lib, x, kind, at, t, keep, 1.5, 3.0, in_place=in_place)
    clean = np.where(np.isnan(x), 0.0, x)
    want = vo.distill(clean, at, t, keep, float(np.float32(1.5)), 3.0)
    assert got["token_loss"][8] == np.inf and got["token_loss"][10] == np.inf and got["loss"] == np.inf
    assert np.isfinite(got["dlogits"]).all() and got["token_loss"][7] == 0
    fine = np.isfinite(want["token_loss"])
    # the infinite losses aside (the mean is infinite), everything is within its bound
    got["loss"], got["token_loss"] = want["loss"], np.where(fine, got["token_loss"], want["token_loss"])
    check_distill(got, clean, kind, at, t, keep, 1.5, 3.0)


def test_distill_not_a_number(cuda_lib):
    x, _, rng = logits_of(4, 300, "f32", seed=23)
    at, t = lists_of(x, 5, rng)
    x[1, 17] = np.nan
    t[2, 0] = np.nan
    got = run_distill(cuda_lib, x, "f32", at, t)
    assert np.isnan(got["token_loss"][1:3]).all() and np.isfinite(got["token_loss"][[0, 3]]).all()
    assert np.isnan(got["dlogits"][1]).all() and np.isfinite(got["dlogits"][[0, 3]]).all()
    other = np.setdiff1d(np.arange(300), at[2])
    assert np.isnan(got["dlogits"][2, at[2]]).all() and np.isfinite(got["dlogits"][2, other]).all()


@pytest.mark.parametrize("T", [0, 5])
def test_distill_nothing_counted(cuda_lib, T):
    x, _, rng = logits_of(max(T, 1), 100, "bf16")
    at, t = lists_of(x, 4, rng)
    at[:, 0] = -1
    got = run_distill(cuda_lib, x[:T], "bf16", at[:T], t[:T])
    assert got["kept"] == 0 and got["loss"] == 0 and (got["token_loss"] == 0).all() and (got["dlogits"] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,k", [(1900, 301, 200), (1900, 2050, 9), (700, 1003, 300)])
def test_distill_many_short_rows(cuda_lib, T, V, k, kind):
    """Small blocks, and lists longer than they are."""
    x, _, rng = logits_of(53, V, kind, seed=29)
    at, t = lists_of(x, k, rng)
    at[7, k // 2:] = at[7, 0]
    at[9, 0] = -1
    pick = np.arange(T) % 53
    n = (pick != 9).sum()
    for grad in (False, True):
        got = run_distill(cuda_lib, x[pick], kind, at[pick], t[pick], tau=0.9, grad=grad)
        assert got["kept"] == n
        one = {"token_loss": got["token_loss"][:53], "kept": 52}
        one["loss"] = vo.distill(x, at, t, None, float(np.float32(0.9)))["loss"]
        if grad:
            assert (got["dlogits"] == got["dlogits"][:53][pick]).all()
            one["dlogits"] = got["dlogits"][:53]
        check_distill(one, x, kind, at, t, None, 0.9, 52 / n)
        mean = got["token_loss"].sum() / n
        assert abs(got["loss"] - mean) <= 2.0**-24 * (T / 128 + 32) * mean


def test_distill_a_share_larger_than_shared_memory(cuda_lib):
    """What a CTA cannot hold it reads again."""
    x, _, rng = logits_of(2, 500003, "f32", seed=30)
    at, t = lists_of(x, 20, rng)
    for in_place in (False, True):
        check_distill(run_distill(cuda_lib, x, "f32", at, t, in_place=in_place), x, "f32", at, t)


def test_distill_longest_lists(cuda_lib):
    x, _, rng = logits_of(3, 2500, "bf16", seed=24)
    at, t = lists_of(x, 1024, rng)
    check_distill(run_distill(cuda_lib, x, "bf16", at, t), x, "bf16", at, t)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind,V", [("bf16", 33003), ("f32", 17001), ("bf16", 81920), ("f32", 70007), ("bf16", 131076)])
def test_distill_many_long_rows(cuda_lib, V, kind, in_place):
    """Enough long rows that an SM takes several: rows that fit its buffers and
    rows that do not, whole chunks and odd ends, rows that do not count between
    them.  Thirteen kinds of row repeat: the first of each is compared with 64
    bits, the others with it."""
    T, kinds, k, tau = 330, 13, 70, 1.4
    x, _, rng = logits_of(kinds, V, kind, seed=26)
    at, t = lists_of(x, k, rng)
    length = rng.integers(1, k + 1, size=kinds)
    length[2] = k
    at[np.arange(k) >= length[:, None]] = V
    at[3, 5:60] = at[3, :55]
    length[3] = 60
    at[3, 60:] = -1
    x[4, V // 2:] = -np.inf
    t[5, :3] = -np.inf
    keep = np.ones(T, np.uint8)
    pick = np.arange(T) % kinds
    at, t = at[pick], t[pick]
    at[pick == 6, 0] = -1
    keep[pick == 7] = 0
    keep[40:100] = 0
    x_all = x[pick]
    x_all[(keep == 0) | (pick == 6)] = np.nan  # never read
    got = run_distill(cuda_lib, x_all, kind, at, t, keep, tau, 2.0, in_place=in_place)
    counted = (keep != 0) & (pick != 6)
    n = counted.sum()
    assert got["kept"] == n
    assert (got["token_loss"][~counted] == 0).all() and (got["dlogits"][~counted] == 0).all()
    one = np.array([np.nonzero(counted & (pick == r))[0][0] for r in range(kinds) if r not in (6, 7)])
    for r in one:
        same = counted & (pick == pick[r])
        assert (got["dlogits"][same] == got["dlogits"][r]).all() and (got["token_loss"][same] == got["token_loss"][r]).all()
    part = {"token_loss": got["token_loss"][one], "dlogits": got["dlogits"][one], "kept": len(one)}
    want = vo.distill(x[pick[one]], at[one], t[one], None, float(np.float32(tau)), 2.0 * len(one) / n)
    part["loss"] = want["loss"]
    check_distill(part, x[pick[one]], kind, at[one], t[one], None, tau, 2.0 * len(one) / n)
    # a masked word in the teacher's list of kind 4: its loss is infinite, and so is the mean
    assert got["token_loss"][pick == 4][0] == np.inf and got["loss"] == np.inf


@pytest.mark.parametrize("k", [1, 3, 255, 256, 257])
def test_distill_many_long_rows_lists(cuda_lib, k):
    """Lists of every length that a list warp takes, and one more."""
    T, kinds, V = 320, 8, 30001
    x, _, rng = logits_of(kinds, V, "bf16", seed=28)
    at, t = lists_of(x, k, rng)
    at[1, k // 2:] = at[1, 0]  # the same index many times
    pick = np.arange(T) % kinds
    got = run_distill(cuda_lib, x[pick], "bf16", at[pick], t[pick])
    for r in range(kinds):
        assert (got["dlogits"][pick == r] == got["dlogits"][r]).all()
    # the first of each as a batch of their own, whose mean's gradient is T / kinds times theirs
    one = {"token_loss": got["token_loss"][:kinds], "dlogits": got["dlogits"][:kinds], "kept": kinds,
           "loss": vo.distill(x, at, t)["loss"]}
    check_distill(one, x, "bf16", at, t, None, 1.0, kinds / T)


def test_distill_expired_wait_is_reported(cuda_lib):
    """The producer withholds its copies: the waits run out, the call reports
    it, and the next one is right."""
    fc = cuda_lib
    x, _, rng = logits_of(310, 33000, "bf16", seed=27)
    at, t = lists_of(x, 8, rng)
    want = run_distill(fc, x, "bf16", at, t)
    mean = want["token_loss"].sum() / 310
    assert abs(want["loss"] - mean) <= 2.0**-24 * (310 / 576 + 32) * mean
    fc.axonn_set_wait_timeout_ns(20_000_000)
    fc.axonn_debug_set_inject(1)
    try:
        with pytest.raises(fc.AxonnError) as e:
            run_distill(fc, x, "bf16", at, t)
        assert e.value.status == fc.ERR_TIMEOUT
    finally:
        fc.axonn_debug_set_inject(0)
        fc.axonn_set_wait_timeout_ns(4_000_000_000)
    again = run_distill(fc, x, "bf16", at, t)
    assert all(np.array_equal(want[n], again[n]) for n in want)


def test_distill_against_differences(cuda_lib):
    """The mean's gradient by differences of the kernel's own loss along random
    directions: step^2 f'''/6, and the loss's error over the step, both below
    1e-3 here."""
    T, V, tau, s = 5, 200, 1.3, 2e-2
    x, _, rng = logits_of(T, V, "f32", seed=25, spread=1.0)
    at, t = lists_of(x, 8, rng)
    d = run_distill(cuda_lib, x, "f32", at, t, tau=tau)["dlogits"]
    for _ in range(6):
        u = rng.normal(size=x.shape)
        u /= np.linalg.norm(u)
        up, down = (run_distill(cuda_lib, stored(x + e * u, "f32"), "f32", at, t, tau=tau, grad=False)["loss"]
                    for e in (s, -s))
        assert abs((up - down) / (2 * s) - (d * u).sum()) < 1e-3


# ------------------------------------------------------------------ all of them, as they are used
def test_teacher_to_student(cuda_lib):
    """A teacher's lists, made by axonn_token_logprobs with its masked rows'
    -1, are what axonn_distill reads; a student equal to its teacher has KL =
    -ln of the list's share, and following the gradient lowers the loss."""
    import torch
    fc = cuda_lib
    T, V, k, tau = 24, 3001, 16, 1.0
    x, _, rng = logits_of(T, V, "bf16", seed=31)
    keep = gpu((rng.random(T) < 0.8).astype(np.uint8))
    teacher = rows_on_gpu(x, "bf16")
    index = torch.empty((T, k), dtype=torch.int32, device="cuda")
    value = torch.empty((T, k), device="cuda")
    fc.axonn_token_logprobs(teacher, top_index=index, top_logprob=value, keep=keep)
    token, loss = torch.empty(T, device="cuda"), torch.empty(1, device="cuda")
    kept = torch.empty(1, dtype=torch.int32, device="cuda")
    fc.axonn_distill(teacher, index, value, token, loss, kept)  # no keep: the lists say it
    fc.axonn_sync_status()
    on = keep.cpu().numpy() != 0
    assert kept.item() == on.sum()
    share = np.exp(vo.token_logprobs(x, None, None, 1.0, k)["top_logprob"]).sum(axis=1)
    assert np.allclose(host(token)[on], -np.log(share[on]), atol=2e-5) and (host(token)[~on] == 0).all()
    student, d = rows_on_gpu(x + rng.normal(size=x.shape), "f32"), rows_on_gpu(x, "f32")
    fc.axonn_distill(student, index, value, token, loss, kept, dlogits=d, temperature=tau)
    first = loss.item()
    student -= d * T
    fc.axonn_distill(student, index, value, token, loss, kept, temperature=tau)
    assert loss.item() < first


def test_policy_step(cuda_lib):
    """Forward and backward as a policy step calls them, against torch's
    autograd in 64 bits on the same logits."""
    import torch
    fc = cuda_lib
    T, V, tau = 50, 2003, 0.9
    x, tokens, rng = logits_of(T, V, "f32", seed=32)
    tokens[::9] = -100
    adv = rng.normal(size=T)
    X, d = rows_on_gpu(x, "f32"), rows_on_gpu(x, "f32")
    lp, H, lse = (torch.empty(T, device="cuda") for _ in range(3))
    fc.axonn_token_logprobs(X, tokens=i32(tokens), logprob=lp, entropy=H, lse=lse, temperature=tau)
    g, h = f32(-adv / T), torch.full((T,), -0.01 / T, device="cuda")
    fc.axonn_token_logprobs_bwd(X, lse, d, tokens=i32(tokens), dlogprob=g, entropy=H, dentropy=h, temperature=tau)
    fc.axonn_sync_status()
    z = torch.from_numpy(x).requires_grad_(True)
    logp = torch.log_softmax(z / float(np.float32(tau)), dim=1)
    inside = torch.from_numpy(tokens >= 0)
    own = logp[torch.arange(T), torch.from_numpy(np.maximum(tokens, 0))]
    ent = torch.special.entr(logp.exp()).sum(1)
    (g.double().cpu() * torch.where(inside, own, 0.0)).sum().add((h.double().cpu() * ent).sum()).backward()
    want = z.grad.numpy()
    assert np.abs(host(d) - want).max() <= 2e-5 * np.abs(want).max()


@pytest.mark.parametrize("T", [1, 3, 200])
def test_in_a_graph_on_another_stream(cuda_lib, T):
    """Captured once and replayed on new inputs, on a stream of its own: as the
    same calls made one by one."""
    import torch
    fc = cuda_lib
    V, k = 5003, 10
    x, tokens, rng = logits_of(T, V, "bf16", seed=41)
    X = rows_on_gpu(x, "bf16")
    tok = i32(tokens)
    lp, H, lse, token = (torch.empty(T, device="cuda") for _ in range(4))
    index, value = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    loss, kept = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    g, h = f32(rng.normal(size=T)), f32(rng.normal(size=T))
    d1, d2 = rows_on_gpu(x, "bf16"), rows_on_gpu(x, "bf16")

    def step():
        fc.axonn_token_logprobs(X, tokens=tok, logprob=lp, entropy=H, lse=lse, top_index=index, top_logprob=value)
        fc.axonn_token_logprobs_bwd(X, lse, d1, tokens=tok, dlogprob=g, entropy=H, dentropy=h)
        fc.axonn_distill(X, index, value, token, loss, kept, dlogits=d2, temperature=2.0)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for seed in (42, 43):
        x, tokens, _ = logits_of(T, V, "bf16", seed=seed)
        X.copy_(rows_on_gpu(x, "bf16"))
        tok.copy_(i32(tokens))
        outs = (lp, H, lse, index, value, d1, token, loss, kept, d2)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [host(o) for o in outs]
        for o in outs:
            o.fill_(1)
        step()
        torch.cuda.synchronize()
        for a, b in zip(replayed, outs):
            assert np.array_equal(a, host(b))


def test_two_streams_at_once(cuda_lib):
    import torch
    fc = cuda_lib
    V, k = 40001, 20
    sides = []
    for seed in (51, 52):
        x, _, rng = logits_of(90, V, "bf16", seed=seed)
        at, t = lists_of(x, k, rng)
        sides.append(dict(X=rows_on_gpu(x, "bf16"), at=i32(at), t=f32(t), d=rows_on_gpu(x, "bf16"),
                          token=torch.empty(90, device="cuda"), loss=torch.empty(1, device="cuda"),
                          kept=torch.empty(1, dtype=torch.int32, device="cuda"),
                          index=torch.empty((90, k), dtype=torch.int32, device="cuda"),
                          value=torch.empty((90, k), device="cuda"), stream=torch.cuda.Stream()))

    def both(s):
        fc.axonn_token_logprobs(s["X"], top_index=s["index"], top_logprob=s["value"], stream=s["stream"])
        fc.axonn_distill(s["X"], s["at"], s["t"], s["token"], s["loss"], s["kept"], dlogits=s["d"], stream=s["stream"])
    names = ("index", "value", "token", "loss", "kept", "d")
    torch.cuda.synchronize()
    alone = []
    for s in sides:
        both(s)
        torch.cuda.synchronize()
        alone.append([host(s[n]) for n in names])
    for _ in range(5):
        for s in sides:
            both(s)
    torch.cuda.synchronize()
    for s, want in zip(sides, alone):
        for n, w in zip(names, want):
            assert np.array_equal(host(s[n]), w), n


def test_offsets_past_32_bits(cuda_lib):
    """Rows that begin beyond 2^31 and 2^32 elements of one buffer."""
    import torch
    fc = cuda_lib
    V, ld = 1003, 1 << 25
    x, tokens, rng = logits_of(130, V, "bf16", seed=61)
    full = torch.empty((130, ld), dtype=torch.bfloat16, device="cuda")
    X = full[:, :V]
    X.copy_(gpu(x).to(torch.bfloat16))
    check = run_logprobs(fc, x, "bf16", tokens, k=6)
    lp, lse = torch.empty(130, device="cuda"), torch.empty(130, device="cuda")
    index = torch.empty((130, 6), dtype=torch.int32, device="cuda")
    fc.axonn_token_logprobs(X, tokens=i32(tokens), logprob=lp, lse=lse, top_index=index)
    assert np.array_equal(host(lp), check["logprob"]) and np.array_equal(host(index), check["top_index"])
    at, t = lists_of(x, 6, rng)
    small = run_distill(fc, x, "bf16", at, t)
    token, loss = torch.empty(130, device="cuda"), torch.empty(1, device="cuda")
    kept = torch.empty(1, dtype=torch.int32, device="cuda")
    g = f32(rng.normal(size=130))
    want = run_backward(fc, x, "bf16", host(lse), tokens, host(g))
    fc.axonn_distill(X, i32(at), f32(t), token, loss, kept, dlogits=X)  # in place
    assert np.array_equal(host(X), small["dlogits"])
    X.copy_(gpu(x).to(torch.bfloat16))
    fc.axonn_token_logprobs_bwd(X, lse, X, tokens=i32(tokens), dlogprob=g)
    assert np.array_equal(host(X), want)


def test_more_rows_than_a_grid_dimension(cuda_lib):
    """70000 rows: the backward's blocks take more than one."""
    x, tokens, rng = logits_of(70000, 16, "f32", seed=71)
    got = run_logprobs(cuda_lib, x, "f32", tokens)
    check_logprobs(got, x, tokens)
    g = rng.normal(size=70000).astype(np.float32)
    lse = got["lse"].astype(np.float32)
    check_backward(run_backward(cuda_lib, x, "f32", lse, tokens, g), x, "f32", lse, tokens, g)


def test_a_row_past_2_31_bytes(cuda_lib):
    """One row of 1.1e9 words, zeros but for a few: closed forms, and offsets in
    bytes past 2^31 in every kernel that takes it."""
    import math

    import torch
    fc = cuda_lib
    V, k = 1_100_000_005, 4
    X = torch.zeros((1, V + 3), dtype=torch.bfloat16, device="cuda")[:, :V]
    places, values = [V - 1, 12, 1_073_741_830, 536_870_921], [24.0, 23.0, 22.0, 21.0]
    for at, v in zip(places, values):
        X[0, at] = v
    lse = math.log(V - k + sum(math.exp(v) for v in values))
    lp, H, out = (torch.empty(1, device="cuda") for _ in range(3))
    index = torch.empty((1, k), dtype=torch.int32, device="cuda")
    value = torch.empty((1, k), device="cuda")
    fc.axonn_token_logprobs(X, tokens=i32([places[2]]), logprob=lp, entropy=H, lse=out, top_index=index,
                            top_logprob=value)
    assert host(index)[0].tolist() == places
    # sums of 1.1e9 terms over 8 x 256 threads: 67138 vectors each, 2^-24 for each
    # addition; the terms are equal, so their roundings may all go one way
    tol = 2.0**-24 * V / (8 * 2048) * 2 + 2.0**-20
    assert abs(host(out)[0] - lse) <= tol and abs(host(lp)[0] - (values[2] - lse)) <= tol
    assert np.abs(host(value)[0] - (np.array(values) - lse)).max() <= tol
    d = torch.full((1, V + 3), 7.0, dtype=torch.bfloat16, device="cuda")[:, :V]
    fc.axonn_token_logprobs_bwd(X, out, d, tokens=i32([places[2]]), dlogprob=f32([1.0]))
    p0 = math.exp(-lse)
    got = host(d[0, torch.tensor([*places, 0, V - 2], device="cuda")])
    want = np.array([-math.exp(v - lse) for v in values] + [-p0, -p0])
    want[2] += 1
    assert (np.abs(got - want) <= (2.0**-8 + 2 * tol) * np.abs(want) + 2 * tol).all()
    assert bool((d[0, 100:200].double() / -p0 - 1).abs().max() <= 2.0**-8 + 2 * tol)
    fc.axonn_distill(X, index, value, lp, H, i32([0]), dlogits=d)
    got = host(d[0, torch.tensor([*places, 0, V - 2], device="cuda")])
    q = np.exp(np.array(values) - 24)
    q = q / q.sum()
    want = np.array([math.exp(v - lse) - w for v, w in zip(values, q)] + [p0, p0])
    assert (np.abs(got - want) <= (2.0**-8 + 2 * tol) * np.abs(want) + 4 * tol * np.append(q, [p0, p0])).all()
    kl = float((q * (np.log(q) - (np.array(values) - lse))).sum())
    assert abs(host(lp)[0] - kl) <= 2 * tol
    assert bool((d._base[:, V:] == 7).all())


def test_no_rows(cuda_lib):
    import torch
    X = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, device="cuda")
    cuda_lib.axonn_token_logprobs(X, lse=none)
    cuda_lib.axonn_token_logprobs_bwd(X, none, X, tokens=none.to(torch.int32), dlogprob=none)
    cuda_lib.axonn_sync_status()


def test_one_row_of_any_stride(cuda_lib):
    """The stride of a single row says nothing: an odd vocabulary as torch
    lays it out."""
    import torch
    x, tokens, _ = logits_of(1, 50257, "bf16", seed=81)
    X = gpu(x).to(torch.bfloat16)
    assert X.stride(0) % 8 != 0
    lse = torch.empty(1, device="cuda")
    cuda_lib.axonn_token_logprobs(X, lse=lse)
    assert host(lse)[0] == run_logprobs(cuda_lib, x, "bf16", tokens)["lse"][0]
