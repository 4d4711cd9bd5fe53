"""The way back through log probabilities for logits of any size, forward then
backward, against a gradient from the logits alone in 64 bits.

Bounds (derived; D, S and E as in test_vocab_gpu).  The parts of lse are the
row's largest logit, exact, and ln S, off by E.  ln p = (x - m) inv - ln S has
roundings of the difference, of inv and of the sum: E + D 2^-23 + |ln p| 2^-24,
and its exponential one of log2(e), one of the product and 2^-22 for the function
unit: p is off by e_p = E + (D + |ln p| + 1) 2^-22 of itself.  H is off by e_H as
the forward's bound has it.
  g ([v = y] - p) - h p (ln p + H):  p (w (e_p + 2^-21) + |h| (e_p + e_H)), with
  w = |g| + |h| (|ln p| + |H|), and |g| 2^-22 (p + [v = y]) for g / tau
and one rounding to the logits' type.  Where p is below 2^-126 it is 0, which
leaves out 2^-126 w.
"""
import numpy as np
import pytest

from oracle import vocab as vo
from test_vocab_gpu import (HALF, TINY, check_logprobs, close, f32, gpu, host, i32, logits_of, numbers,
                            padding_untouched, rows_on_gpu, run_backward, run_logprobs, special_rows, stored)

pytestmark = pytest.mark.gpu


def step(fc, x, kind, tokens, g=None, h=None, keep=None, tau=1.0, in_place=False):
    """Forward with lse in parts, then backward; what both leave."""
    import torch
    T = x.shape[0]
    X = rows_on_gpu(x, kind)
    keep = None if keep is None else gpu(keep.astype(np.uint8))
    lp, H = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    lse = torch.full((T, 2), 7.0, device="cuda")
    fc.axonn_token_logprobs(X, tokens=i32(tokens), logprob=lp, entropy=H, lse=lse, keep=keep, temperature=tau)
    out = X if in_place else rows_on_gpu(np.full(x.shape, 7.0), kind)
    fc.axonn_token_logprobs_bwd(X, lse, out, tokens=None if g is None else i32(tokens),
                                dlogprob=None if g is None else f32(g), entropy=None if h is None else H,
                                dentropy=None if h is None else f32(h), keep=keep, temperature=tau)
    fc.axonn_sync_status()
    assert padding_untouched(out)
    return host(lse), host(out)


def check_step(got, x, kind, tokens, g=None, h=None, tau=1.0):
    """Rows of finite logits and -inf."""
    T, V = x.shape
    tau = float(np.float32(tau))
    lse, d = got
    D, p, lnS, pD, E = numbers(x, tau)
    empty = (x == -np.inf).all(axis=1)
    assert np.array_equal(lse[:, 0], x.max(axis=1))
    close(lse[:, 1], np.where(empty, -np.inf, lnS), np.where(empty, 0, E), "ln S")
    want = vo.policy_gradient(x, tokens, g, h, tau)
    lp = np.where((p > 0) & ~empty[:, None], np.abs(vo.log_softmax(x, tau)), 0.0)
    D = np.where(p > 0, D, 0.0)
    H = -np.where(p > 0, -p * lp, 0.0).sum(axis=1)[:, None]
    eH = (E * (1 + pD) + 2.0**-22 * ((p * D * (D + 2)).sum(axis=1) + lnS + pD))[:, None]
    ep = E[:, None] + (D + lp + 1) * 2.0**-22
    G = np.zeros((T, 1)) if g is None else np.where((tokens >= 0) & (tokens < V), np.abs(np.float64(g)), 0.0)[:, None]
    hh = np.zeros((T, 1)) if h is None else np.abs(np.float64(h))[:, None]
    w = G + hh * (lp + H)
    tol = p * (w * (ep + 2.0**-21) + hh * (ep + eH)) + G * 2.0**-22 * (p + (np.arange(V) == tokens[:, None]))
    tol = np.where(empty[:, None], 0.0, (tol + 2.0**-126 * (w + 256 * hh)) / tau + HALF[kind] * np.abs(want) + TINY)
    close(d, want, tol, "dlogits")
    # the gradient of ln p and of H does not move a row's mean
    assert (np.abs(d.sum(axis=1)) <= tol.sum(axis=1)).all()


@pytest.mark.parametrize("tau", [1.0, 0.7, 1e-3, 30.0])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [8, 1003, 8200])
def test_special_rows(cuda_lib, V, kind, tau):
    """Masks of the type's lowest value throughout, constant, huge and far rows."""
    names, x = special_rows(V, kind)
    extra = np.stack([np.full(V, -1e9), np.where(np.arange(V) % 3 == 0, -1e9, -1e9 - 1e7), np.full(V, 1e6),
                      np.random.default_rng(4).normal(size=V) * 4 + 1e6])
    names, x = names + ["masked", "masked in two steps", "high", "high, spread"], np.concatenate([x, stored(extra, kind)])
    T = len(names)
    rng = np.random.default_rng(8)
    tokens, g, h = np.full(T, V // 2), rng.normal(size=T), rng.normal(size=T)
    tokens[::5] = V - 1
    g, h = np.float64(np.float32(g)), np.float64(np.float32(h))
    number = ~(np.isnan(x) | (x == np.inf)).any(axis=1)
    for kw in (dict(g=g), dict(h=h), dict(g=g, h=h)):
        lse, d = step(cuda_lib, x, kind, tokens, tau=tau, **kw)
        assert np.isnan(d[~number]).all(), [n for n, ok in zip(names, number) if not ok]
        part = {n: v[number] for n, v in kw.items()}
        check_step((lse[number], d[number]), x[number], kind, tokens[number], tau=tau, **part)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (1, 7), (2, 9), (5, 130), (3, 4099), (170, 600), (1, 131075)])
def test_sizes(cuda_lib, T, V, kind, in_place):
    x, tokens, rng = logits_of(T, V, kind, seed=14)
    g, h = np.float64(np.float32(rng.normal(size=T))), np.float64(np.float32(rng.normal(size=T)))
    if T > 2:
        tokens[1], x[2] = -100, -1e9
        x[2] = stored(x[2], kind)
    for kw in (dict(g=g), dict(h=h), dict(g=g, h=h)):
        check_step(step(cuda_lib, x, kind, tokens, tau=0.8, in_place=in_place, **kw), x, kind, tokens, tau=0.8, **kw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_left_out(cuda_lib, kind):
    """Zeros, whatever is in them: in lse, too."""
    x, tokens, rng = logits_of(12, 500, kind, seed=15)
    keep = (np.arange(12) % 3 != 0).astype(np.uint8)
    g = np.float64(np.float32(rng.normal(size=12)))
    g[4] = 0
    x[0], x[3, 7], x[4, 9] = -np.inf, np.nan, np.nan
    lse, d = step(cuda_lib, x, kind, tokens, g=g, keep=keep)
    off = keep == 0
    assert (lse[off] == 0).all() and (d[off] == 0).all() and (d[4] == 0).all()
    on = ~off & (np.arange(12) != 4)
    check_step((lse[on], d[on]), x[on], kind, tokens[on], g=g[on])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_lse_in_one_number(cuda_lib, kind):
    """What one fp32 number cannot tell a gradient from is NaN; in one or in
    parts, ordinary rows differ by lse's rounding."""
    V = 700
    low = special_rows(8, kind)[1][1, 0]
    x, tokens, _ = logits_of(8, V, kind, seed=17)
    x[1], x[2], x[3], x[4] = low, -1e9, 7e4, -np.inf
    x[5, :] = 65000.0
    x[6, ::2] = -np.inf
    x[6, tokens[6]] = 1.0
    x = stored(x, kind)
    g = np.ones(8)
    for tau in (1.0, 0.5):
        with np.errstate(over="ignore"):
            lse = vo.logsumexp(x, tau).astype(np.float32)
        got = run_backward(cuda_lib, x, kind, lse, tokens, g, tau=tau)
        far = np.abs(lse.astype(np.float64)) > 65536
        assert far[1:4].all() and far[4] and far[5] == (tau == 0.5)
        far[4] = False
        assert np.isnan(got[far]).all() and (got[4] == 0).all()
        want = vo.policy_gradient(x, tokens, g, None, tau)
        fine = ~far
        tol = np.where(x[fine] > -np.inf, 2.0**-23 * np.abs(lse[fine].astype(np.float64))[:, None], 0) + 2.0**-18
        tol[x[fine].max(axis=1) == -np.inf] = 0
        close(got[fine], want[fine], (tol + HALF[kind]) * (np.abs(want[fine]) + 1.0) / tau, "one number")
    # below fp32's range, some words without a probability
    x[1, ::2] = -np.inf
    lse = np.full(8, -np.inf)
    got = run_backward(cuda_lib, x, kind, lse, tokens, g, tau=0.5, in_place=True)
    assert np.isnan(got[1, 1::2]).all() and (got[1, ::2] == 0).all()


def test_in_a_graph(cuda_lib):
    import torch
    fc = cuda_lib
    T, V = 40, 3001
    x, tokens, rng = logits_of(T, V, "bf16", seed=18)
    X, tok, g = rows_on_gpu(x, "bf16"), i32(tokens), f32(rng.normal(size=T))
    lse, lp, d = torch.empty((T, 2), device="cuda"), torch.empty(T, device="cuda"), rows_on_gpu(x, "bf16")

    def both():
        fc.axonn_token_logprobs(X, tokens=tok, logprob=lp, lse=lse)
        fc.axonn_token_logprobs_bwd(X, lse, d, tokens=tok, dlogprob=g)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for shift in (0.0, -1e9):
        X.copy_(rows_on_gpu(x + shift, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [host(t) for t in (lse, lp, d)]
        for t in (lse, lp, d):
            t.fill_(1)
        both()
        torch.cuda.synchronize()
        assert all(np.array_equal(a, host(b)) for a, b in zip(replayed, (lse, lp, d)))


@pytest.mark.parametrize("tau", [0.5, 1.0, 1.5, 3.0, 1e4])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_finite_logits_further_apart_than_fp32_reaches(cuda_lib, kind, tau):
    """ln p is -inf only where it is beyond fp32 itself, in shares of a row (one
    row), too; with a NaN or an infinity beside them it is NaN."""
    low = special_rows(8, kind)[1][1, 0]
    for T, V in ((40, 300), (1, 70001)):
        x = stored(np.full((T, V), low), kind)
        x[:, ::3], x[:, 7] = -low, -np.inf
        x[:, 5] = 0.0
        tokens = np.array([1, 0, 5, 7])[np.arange(T) % 4]
        if T > 1:
            x[8, 20], x[9, 20] = np.nan, np.inf
            x[10] = np.where(np.arange(V) % 4 == 1, low, -np.inf)
            x[11] = stored(np.where(np.arange(V) % 4 == 1, low, low / 2), kind)
        got = run_logprobs(cuda_lib, x, kind, tokens, tau=tau, k=min(V, 128))
        fine = ~(np.isnan(x) | (x == np.inf)).any(axis=1)
        assert np.isnan(got["logprob"][~fine]).all() and np.isnan(got["top_logprob"][~fine]).all()
        check_logprobs({n: v[fine] for n, v in got.items()}, x[fine], tokens[fine], tau=tau, k=min(V, 128))
        # beyond fp32 at a temperature of 1, within at 3
        one = np.nonzero(fine & (tokens == 1))[0][0]
        assert (got["logprob"][one] == -np.inf) == (tau < 2)
