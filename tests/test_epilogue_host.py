"""The operators around a layer's products, without a GPU: the 64-bit forms
against published vectors and differences, and every refusal of the entry
points (which comes before any device work)."""
import ctypes

import numpy as np
import pytest

from oracle import epilogue as ep

FAKE = 0x10000000  # never dereferenced


@pytest.fixture(scope="module")
def fc():
    from pmm_fc_layer_gb300 import build as _build
    _build.build()
    import pmm_fc_layer_gb300 as mod
    mod.load()
    return mod


@pytest.mark.parametrize("counter,key,expect", [
    # the generator's published known-answer vectors (ten rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, expect):
    assert tuple(int(w) for w in ep.philox4x32_10(counter, key)) == expect


def test_keep_mask_rate_and_rows():
    keep, scale = ep.keep_mask(64, 1001, 0.25, 5, 9)
    n = keep.size
    assert abs(keep.mean() - 0.75) < 5 * (0.25 * 0.75 / n) ** 0.5   # five standard deviations
    assert scale == np.float32(4 / 3)
    part, _ = ep.keep_mask(3, 8, 0.25, 5, 9)
    assert np.array_equal(part, keep[:3, :8])       # a row's mask does not depend on the extents
    other, _ = ep.keep_mask(64, 1001, 0.25, 5, 10)
    assert (other != keep).mean() > 0.3


@pytest.mark.parametrize("name", ep.ACTS)
def test_slopes_against_differences(name):
    z = np.linspace(-6, 6, 241) + 0.013
    h = 1e-5
    diff = (ep.act(z + h, name) - ep.act(z - h, name)) / (2 * h)
    assert np.abs(diff - ep.slope(z, name)).max() < 1e-8  # h^2 f'''/6 + eps/h


def test_linear_ce_against_differences():
    rng = np.random.default_rng(3)
    X, W = rng.normal(size=(5, 4)), rng.normal(size=(4, 7))
    y = np.array([2, -1, 6, 0, 9])
    keep = np.array([1, 1, 1, 0, 1])
    r = ep.linear_ce(X, W, y, keep, 2.5)
    assert r["n"] == 2
    h = 1e-6
    for M, name in ((X, "dX"), (W, "dW")):
        for at in np.ndindex(*M.shape):
            old = M[at]
            M[at] = old + h
            up = ep.linear_ce(X, W, y, keep)["loss"]
            M[at] = old - h
            down = ep.linear_ce(X, W, y, keep)["loss"]
            M[at] = old
            assert abs(2.5 * (up - down) / (2 * h) - r[name][at]) < 1e-7


# ------------------------------------------------------------------ refusals
def epi(fc, **kw):
    e = fc.Epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def call_fwd(fc, e, shape=(64, 64, 64), grid=(1, 1, 1), flags=0, X=FAKE, W=FAKE, Y=FAKE, ld=(64, 64, 64)):
    s = fc.Shape(*shape, grid)
    return fc.load().axonn_fc_fwd_epi(X, W, Y, *ld, ctypes.byref(s), flags,
                                      ctypes.byref(e) if e is not None else None, 0)


def call_dgrad(fc, e, flags=0, ws=0, ws_bytes=0, shape=(64, 64, 64)):
    s = fc.Shape(*shape)
    return fc.load().axonn_fc_dgrad_epi(FAKE, FAKE, FAKE, 64, 64, 64, ctypes.byref(s), flags,
                                        ctypes.byref(e), ws, ws_bytes, 0)


@pytest.mark.parametrize("fields,kw,expect", [
    (None, {}, 1),
    (dict(act=5), {}, 1),
    (dict(act=-1), {}, 1),
    (dict(p=-0.1), {}, 1),
    (dict(p=1.5), {}, 1),
    (dict(p=float("nan")), {}, 1),
    (dict(p=0.5), {}, 1),                               # no rng
    (dict(p=0.5, rng=FAKE + 4), {}, 2),
    (dict(bias=FAKE + 2), {}, 2),
    (dict(dbias=FAKE), {}, 1),
    (dict(pre=FAKE, ld_pre=32), {}, 1),
    (dict(pre=FAKE, ld_pre=68), {}, 2),
    (dict(residual=FAKE + 8, ld_residual=64), {}, 2),
    (dict(residual=FAKE, ld_residual=66), dict(flags=0x20), 2),
    ({}, dict(flags=0x4), 1),                           # accumulation does not apply
    ({}, dict(flags=0x8), 1),
    ({}, dict(flags=0x400), 1),
    ({}, dict(grid=(2, 1, 1)), 3),
    ({}, dict(shape=(-1, 64, 64)), 1),
    ({}, dict(X=0), 1),
    ({}, dict(X=FAKE + 8), 2),
    ({}, dict(Y=0), 1),
    ({}, dict(ld=(64, 64, 63)), 1),
    ({}, dict(ld=(64, 68, 64)), 2),
])
def test_forward_refusals(fc, fields, kw, expect):
    e = None if fields is None else epi(fc, **fields)
    assert call_fwd(fc, e, **kw) == expect, fc.axonn_last_error()
    assert fc.axonn_last_error()


@pytest.mark.parametrize("fields,kw,expect", [
    (dict(act=1), {}, 1),                               # the slope needs pre
    (dict(act=1, pre=FAKE + 8, ld_pre=64), {}, 2),
    (dict(bias=FAKE), {}, 1),
    (dict(dbias=FAKE), {}, 4),
    (dict(dbias=FAKE), dict(ws=FAKE, ws_bytes=2 * 64 * 4 - 1), 4),
    (dict(dbias=FAKE), dict(ws=FAKE + 4, ws_bytes=1 << 20), 2),
    (dict(dbias=FAKE + 4), dict(ws=FAKE, ws_bytes=1 << 20), 2),
    ({}, dict(flags=0x200), 1),
])
def test_dgrad_refusals(fc, fields, kw, expect):
    assert call_dgrad(fc, epi(fc, **fields), **kw) == expect, fc.axonn_last_error()


@pytest.mark.parametrize("fields,args,expect", [
    (dict(act=2), {}, 1),
    (dict(bias=FAKE), {}, 1),
    (dict(residual=FAKE), {}, 1),
    (dict(), dict(flags=0x20), 1),
    (dict(), dict(rows=-1), 1),
    (dict(), dict(cols=1 << 31), 3),
    (dict(), dict(lddy=60), 1),
    (dict(), dict(lddz=68), 2),
    (dict(dbias=FAKE), {}, 4),
])
def test_elementwise_backward_refusals(fc, fields, args, expect):
    a = dict(lddy=64, lddz=64, rows=64, cols=64, flags=0)
    a.update(args)
    st = fc.load().axonn_epi_bwd(FAKE, a["lddy"], FAKE, a["lddz"], a["rows"], a["cols"], a["flags"],
                                 ctypes.byref(epi(fc, **fields)), 0, 0, 0)
    assert st == expect, fc.axonn_last_error()


@pytest.mark.parametrize("args,expect", [
    (dict(p=2.0), 1), (dict(rng=0), 1), (dict(x=0), 1), (dict(x=FAKE + 2), 2), (dict(ldx=32), 1),
    (dict(ldy=65), 2), (dict(res=FAKE, ldr=60), 1), (dict(flags=0x20), 1), (dict(rows=-2), 1),
])
def test_dropout_refusals(fc, args, expect):
    a = dict(x=FAKE, ldx=64, res=0, ldr=0, y=FAKE, ldy=64, rows=8, cols=64, p=0.5, rng=FAKE, flags=0)
    a.update(args)
    st = fc.load().axonn_dropout(a["x"], a["ldx"], a["res"], a["ldr"], a["y"], a["ldy"], a["rows"],
                                 a["cols"], a["p"], a["rng"], a["flags"], 0)
    assert st == expect, fc.axonn_last_error()


@pytest.mark.parametrize("args,expect", [
    (dict(V=0), 1), (dict(T=-1), 1), (dict(flags=0x24), 1), (dict(flags=0x1), 1), (dict(loss=0), 1),
    (dict(labels=0), 1), (dict(X=0), 1), (dict(X=FAKE + 8), 2), (dict(ldw=60), 1), (dict(ldw=100), 2),
    (dict(dX=FAKE, lddx=32), 1), (dict(dW=FAKE, lddw=100), 2), (dict(ws=0), 4), (dict(ws_bytes=100), 4),
    (dict(ws=FAKE + 16), 2), (dict(V=1 << 31), 3),
])
def test_linear_ce_refusals(fc, args, expect):
    a = dict(X=FAKE, ldx=64, W=FAKE, ldw=104, labels=FAKE, T=16, K=64, V=100, flags=0, loss=FAKE, dX=0,
             lddx=64, dW=0, lddw=104, ws=FAKE, ws_bytes=1 << 30)
    a.update(args)
    st = fc.load().axonn_linear_ce(a["X"], a["ldx"], a["W"], a["ldw"], a["labels"], 0, a["T"], a["K"],
                                   a["V"], 1.0, a["flags"], FAKE, 0, a["loss"], FAKE, a["dX"], a["lddx"],
                                   a["dW"], a["lddw"], a["ws"], a["ws_bytes"], 0)
    assert st == expect, fc.axonn_last_error()


def test_workspace_sizes(fc):
    assert fc.axonn_epi_workspace_size(33, 10) == 2 * 16 * 4
    assert fc.axonn_epi_workspace_size(0, 10) == 0
    T, K, V = 4096, 512, 128256
    loss = fc.axonn_linear_ce_workspace_size(T, K, V, grad=False)
    whole = fc.axonn_linear_ce_workspace_size(T, K, V)
    # all of P in one piece, and dX as the fp32 parts of a split reduction, if any
    assert 2 * T * V <= whole - loss <= 2 * T * V + 16 * 4 * T * K
    piece = fc.axonn_linear_ce_workspace_size(T, K, V, piece=8192)
    assert piece - loss == 2 * T * 8192 + 4 * T * K   # a piece, and dX's fp32 sum
    assert fc.axonn_linear_ce_workspace_size(T, K, V, piece=8191) == piece
    big = fc.axonn_linear_ce_workspace_size(1 << 20, K, V)
    assert big - fc.axonn_linear_ce_workspace_size(1 << 20, K, V, grad=False) < (3 << 30) + (1 << 20) * 4 * K
    with pytest.raises(fc.AxonnError):
        fc.axonn_linear_ce_workspace_size(T, K, V, piece=-1)


def test_binding_checks(fc):
    import torch
    X = torch.zeros(8, 8, dtype=torch.float16)
    with pytest.raises(ValueError):
        fc.axonn_fc_fwd_epi(X, X, X, fc.Shape(8, 8, 8), stream=0)
    B = torch.zeros(8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fc.axonn_fc_fwd_epi(B, B, B, fc.Shape(8, 8, 8), act="tanh", stream=0)
    with pytest.raises(ValueError):
        fc.axonn_fc_fwd_epi(B, B, B, fc.Shape(8, 8, 8), bias=torch.zeros(4), stream=0)
    with pytest.raises(ValueError):
        fc.axonn_dropout(B, B, 0.5, torch.zeros(2), stream=0)
    with pytest.raises(ValueError):
        fc.axonn_epi_bwd(B, B.float(), stream=0)


class Elsewhere:
    """A tensor's face, without its memory on the device: everything but the
    device is as a call wants it."""

    def __init__(self, shape, kind, device="cpu"):
        import torch
        self.t = torch.zeros(shape, dtype=getattr(torch, kind))
        self.is_cuda = device == "cuda"

    def is_pinned(self):
        return False

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("host", ["X", "W", "Y", "bias", "pre", "residual", "rng"])
def test_host_memory_is_refused_forward(fc, host):
    m = lambda n, shape, kind: Elsewhere(shape, kind, "cpu" if n == host else "cuda")  # noqa: E731
    b = "bfloat16"
    with pytest.raises(ValueError, match=f"{host} must be on the device"):
        fc.axonn_fc_fwd_epi(m("X", (8, 8), b), m("W", (8, 8), b), m("Y", (8, 8), b), fc.Shape(8, 8, 8),
                            bias=m("bias", (8,), "float32"), pre=m("pre", (8, 8), b),
                            residual=m("residual", (8, 8), b), p=0.5, rng=m("rng", (2,), "int64"), stream=0)


@pytest.mark.parametrize("host", ["dY", "W", "dX", "pre", "dbias", "ws"])
def test_host_memory_is_refused_backward(fc, host):
    m = lambda n, shape, kind: Elsewhere(shape, kind, "cpu" if n == host else "cuda")  # noqa: E731
    b = "bfloat16"
    with pytest.raises(ValueError, match=f"{host} must be on the device"):
        fc.axonn_fc_dgrad_epi(m("dY", (8, 8), b), m("W", (8, 8), b), m("dX", (8, 8), b), fc.Shape(8, 8, 8),
                              pre=m("pre", (8, 8), b), act="gelu", dbias=m("dbias", (8,), "float32"),
                              ws=m("ws", (64,), "uint8"), stream=0)
    if host in ("dY", "pre", "dbias", "ws"):
        with pytest.raises(ValueError, match=f"{host} must be on the device"):
            fc.axonn_epi_bwd(m("dY", (8, 8), b), m("dZ", (8, 8), b), pre=m("pre", (8, 8), b), act="gelu",
                             dbias=m("dbias", (8,), "float32"), ws=m("ws", (64,), "uint8"), stream=0)


@pytest.mark.parametrize("host", ["X", "W", "labels", "keep", "token_loss", "lse", "loss", "kept", "dX", "dW", "ws"])
def test_host_memory_is_refused_linear_ce(fc, host):
    m = lambda n, shape, kind: Elsewhere(shape, kind, "cpu" if n == host else "cuda")  # noqa: E731
    b, f = "bfloat16", "float32"
    with pytest.raises(ValueError, match=f"{host} must be on the device"):
        fc.axonn_linear_ce(m("X", (8, 8), b), m("W", (8, 16), b), m("labels", (8,), "int32"),
                           m("token_loss", (8,), f), m("loss", (1,), f), m("kept", (1,), "int32"),
                           m("ws", (1 << 20,), "uint8"), keep=m("keep", (8,), "uint8"), lse=m("lse", (8,), f),
                           dX=m("dX", (8, 8), b), dW=m("dW", (8, 16), b), stream=0)
