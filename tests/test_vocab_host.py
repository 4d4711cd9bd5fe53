"""The operators over rows of vocabulary logits, without a GPU: the 64-bit
forms against torch and differences, and every refusal of the entry points
(which comes before any device work)."""
import numpy as np
import pytest

from oracle import vocab as vo

FAKE = 0x10000000  # never dereferenced


@pytest.fixture(scope="module")
def fc():
    from pmm_fc_layer_gb300 import build as _build
    _build.build()
    import pmm_fc_layer_gb300 as mod
    mod.load()
    return mod


# ------------------------------------------------------------------ the 64-bit forms
@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0])
def test_logprobs_against_torch(tau):
    import torch
    rng = np.random.default_rng(1)
    x = rng.normal(size=(6, 50)) * 3
    x[1, 10:] = -np.inf
    x[2] = np.round(x[2])  # ties
    tokens = np.array([3, 5, -100, 49, 50, 0])
    got = vo.token_logprobs(x, tokens, np.array([1, 1, 1, 1, 1, 0]), tau, 7)
    z = torch.from_numpy(x) / tau
    logp = torch.log_softmax(z, dim=1).numpy()
    want = [logp[0, 3], logp[1, 5], 0, logp[3, 49], 0, 0]
    assert np.allclose(got["logprob"], want, rtol=1e-13, atol=0)
    ent = torch.special.entr(torch.softmax(z, dim=1)).sum(1).numpy()
    assert np.allclose(got["entropy"][:5], ent[:5], rtol=1e-12) and got["entropy"][5] == 0
    assert np.allclose(got["lse"][:5], torch.logsumexp(z, 1).numpy()[:5], rtol=1e-13) and got["lse"][5] == 0
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :7].numpy()
    assert np.array_equal(got["top_index"][:5], order[:5]) and (got["top_index"][5] == -1).all()
    assert np.allclose(got["top_logprob"][:5], np.take_along_axis(logp, order, 1)[:5], rtol=1e-13)


def test_rows_without_a_distribution():
    x = np.array([[-np.inf, -np.inf], [np.nan, 1.0], [np.inf, 0.0], [0.0, -0.0]])
    got = vo.token_logprobs(x, np.array([0, 1, 1, 1]), None, 1.0, 2)
    assert got["lse"][0] == got["logprob"][0] == -np.inf and got["entropy"][0] == 0
    assert np.isnan(got["lse"][1:3]).all() and np.isnan(got["entropy"][1:3]).all()
    assert np.array_equal(got["top_index"], [[0, 1], [0, 1], [0, 1], [0, 1]])


@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_logprobs_backward_against_differences(tau):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(4, 6))
    tokens = np.array([2, -1, 5, 0])
    keep = np.array([1, 1, 1, 0])
    g, h = rng.normal(size=4), rng.normal(size=4)
    f = vo.token_logprobs(x, tokens, keep, tau)
    d = vo.token_logprobs_bwd(x, f["lse"], tokens, g, f["entropy"], h, keep, tau)

    def value():
        r = vo.token_logprobs(x, tokens, keep, tau)
        return (g * r["logprob"] + h * r["entropy"]).sum()
    step = 1e-5
    for at in np.ndindex(*x.shape):
        old = x[at]
        x[at] = old + step
        up = value()
        x[at] = old - step
        down = value()
        x[at] = old
        assert abs((up - down) / (2 * step) - d[at]) < 1e-8  # step^2 f'''/6, and 1e-16 / step


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_against_differences_and_torch(tau):
    import torch
    rng = np.random.default_rng(3)
    x = rng.normal(size=(6, 9))
    at = np.array([[1, 4, 7], [3, 3, 0], [8, -1, 2], [-1, 0, 1], [5, 6, 9], [0, 1, 2]])
    t = rng.normal(size=(6, 3))
    t[4, 1] = -np.inf
    keep = np.array([1, 1, 1, 1, 1, 0])
    r = vo.distill(x, at, t, keep, tau, 1.5)
    assert r["n"] == 4 and np.array_equal(r["counted"], [1, 1, 1, 0, 1, 0])
    # row 0 in torch's own words
    q = torch.softmax(torch.from_numpy(t[0]) / tau, 0)
    logp = torch.log_softmax(torch.from_numpy(x[0]) / tau, 0)[at[0]]
    kl = torch.nn.functional.kl_div(logp, q, reduction="sum")
    assert abs(r["token_loss"][0] - float(kl) * tau**2) < 1e-13
    # lists of one entry: cross entropy at the temperature
    assert abs(r["token_loss"][2] + tau**2 * vo.log_softmax(x, tau)[2, 8]) < 1e-13
    step = 1e-5
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + step
        up = vo.distill(x, at, t, keep, tau)["loss"]
        x[i] = old - step
        down = vo.distill(x, at, t, keep, tau)["loss"]
        x[i] = old
        assert abs(1.5 * (up - down) / (2 * step) - r["dlogits"][i]) < 1e-8


# ------------------------------------------------------------------ refusals
LOG = dict(logits=FAKE, ld=64, tokens=FAKE, keep=0, T=4, V=60, tau=1.0, flags=0, logprob=FAKE, entropy=0, lse=0,
           top_index=0, top_logprob=0, ld_top=0, k=0)
BWD = dict(logits=FAKE, ld=64, tokens=FAKE, keep=0, T=4, V=60, tau=1.0, flags=0, lse=FAKE, dlogprob=FAKE, entropy=0,
           dentropy=0, dlogits=FAKE, ld_d=64)
DIS = dict(logits=FAKE, ld=64, top_index=FAKE, top_logit=FAKE, ld_top=8, keep=0, T=4, V=60, tau=1.0, flags=0,
           token_loss=FAKE, loss=FAKE, kept=FAKE, dlogits=FAKE, ld_d=64, scale=1.0, k=8)
COMMON = [
    (dict(V=0), 1), (dict(V=-1), 1), (dict(T=-1), 1), (dict(T=1 << 31), 3), (dict(V=1 << 31, ld=1 << 31), 3),
    (dict(tau=0.0), 1), (dict(tau=-1.0), 1), (dict(tau=float("nan")), 1), (dict(tau=float("inf")), 1),
    (dict(tau=1e-5), 1), (dict(tau=1e5), 1), (dict(flags=0x20), 1), (dict(flags=0x2), 1),
    (dict(logits=0), 1), (dict(logits=FAKE + 8), 2), (dict(ld=56), 1), (dict(ld=68), 2),
    (dict(flags=0x400, ld=62), 2), (dict(ld=1 << 40), 3),
]


def refuse(fc, fn, base, change, expect):
    packed = {"axonn_token_logprobs": fc._TOKEN_LOGPROBS, "axonn_token_logprobs_bwd": fc._TOKEN_LOGPROBS_BWD,
              "axonn_distill": fc._DISTILL}[fn].pack(*{**base, **change}.values())
    st = getattr(fc.load(), fn)(packed, 0)
    assert st == expect, (change, fc.axonn_last_error())
    assert fc.axonn_last_error()


@pytest.mark.parametrize("fn,base", [("axonn_token_logprobs", LOG), ("axonn_token_logprobs_bwd", BWD),
                                     ("axonn_distill", DIS)])
@pytest.mark.parametrize("change,expect", COMMON)
def test_common_refusals(fc, fn, base, change, expect):
    refuse(fc, fn, base, change, expect)


def test_packed_arguments_are_the_header_s_structs(fc, tmp_path):
    """Sizes and offsets of the packed structs, against the C compiler's."""
    import os
    import subprocess
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    lasts = [("axonn_token_logprobs_t", "k", fc._TOKEN_LOGPROBS, "i4x"), ("axonn_token_logprobs_t", "logprob", None, 56),
             ("axonn_token_logprobs_bwd_t", "ld_dlogits", fc._TOKEN_LOGPROBS_BWD, "q"),
             ("axonn_token_logprobs_bwd_t", "lse", None, 56),
             ("axonn_distill_t", "k", fc._DISTILL, "i"), ("axonn_distill_t", "token_loss", None, 72)]
    body = "".join(f'printf("%zu %zu\\n", sizeof({t}), offsetof({t}, {f}));' for t, f, _, _ in lasts)
    src = tmp_path / "sizes.c"
    src.write_text(f'#include <stdio.h>\n#include "axonn_fc.h"\nint main(void) {{{body} return 0;}}\n')
    subprocess.check_call(["gcc", "-I", include, "-I", cuda, str(src), "-o", str(tmp_path / "sizes")])
    out = subprocess.check_output([str(tmp_path / "sizes")], text=True).split()
    for (t, f, packed, tail), size, at in zip(lasts, map(int, out[::2]), map(int, out[1::2])):
        if packed is None:
            assert at == tail, (t, f)
        else:
            assert size == packed.size, t
            import struct
            assert at == packed.size - struct.calcsize(tail), (t, f)


@pytest.mark.parametrize("fn", ["axonn_token_logprobs", "axonn_token_logprobs_bwd", "axonn_distill"])
def test_null_arguments(fc, fn):
    assert getattr(fc.load(), fn)(None, 0) == 1


@pytest.mark.parametrize("change,expect", [
    (dict(tokens=0), 1), (dict(logprob=0), 1), (dict(tokens=0, logprob=0), 1),
    (dict(k=-1), 1), (dict(k=61, top_index=FAKE, ld_top=61), 1),
    (dict(V=1000, ld=1000, k=129, top_index=FAKE, ld_top=129), 3),
    (dict(top_index=FAKE), 1), (dict(top_logprob=FAKE), 1), (dict(k=2, ld_top=2), 1),
    (dict(k=8, top_index=FAKE, ld_top=7), 1),
])
def test_logprobs_refusals(fc, change, expect):
    refuse(fc, "axonn_token_logprobs", LOG, change, expect)


@pytest.mark.parametrize("change,expect", [
    (dict(lse=0), 1), (dict(tokens=0), 1), (dict(dlogprob=0), 1), (dict(entropy=FAKE), 1), (dict(dentropy=FAKE), 1),
    (dict(tokens=0, dlogprob=0), 1), (dict(dlogits=0), 1), (dict(dlogits=FAKE + 4), 2), (dict(ld_d=68), 2),
    (dict(ld_d=56), 1), (dict(ld_d=72), 1),  # in place with another leading dimension
])
def test_backward_refusals(fc, change, expect):
    refuse(fc, "axonn_token_logprobs_bwd", BWD, change, expect)


@pytest.mark.parametrize("change,expect", [
    (dict(top_index=0), 1), (dict(top_logit=0), 1), (dict(token_loss=0), 1), (dict(loss=0), 1), (dict(kept=0), 1),
    (dict(k=0), 1), (dict(k=-3), 1), (dict(k=1025, ld_top=1025), 3), (dict(ld_top=7), 1),
    (dict(dlogits=FAKE + 2), 2), (dict(ld_d=60), 2), (dict(ld_d=72), 1),
])
def test_distill_refusals(fc, change, expect):
    refuse(fc, "axonn_distill", DIS, change, expect)


class At:
    """A tensor of some device, type, shape and strides, as far as the binding
    looks before the call."""

    def __init__(self, shape, dtype, device=0, stride=None):
        import torch
        self.shape, self.at = torch.Size(shape), device
        self.dtype = getattr(torch, dtype)
        full = torch.empty(shape, device="meta") if stride is None else torch.empty_strided(shape, stride, device="meta")
        self.strides, self.whole = full.stride(), full.is_contiguous()
        self.device = f"cuda:{device}" if device >= 0 else "cpu"

    def get_device(self):
        return self.at

    def stride(self):
        return self.strides

    def is_contiguous(self):
        return self.whole

    def data_ptr(self):
        return FAKE


@pytest.fixture
def on_device_0(fc, monkeypatch):
    """The checks as on device 0; a call that gets past them says so."""
    class Past(Exception):
        pass

    class Library:
        def __getattr__(self, name):
            def call(*args):
                raise Past(name)
            return call
    monkeypatch.setattr(fc, "_current_device", lambda: 0)
    monkeypatch.setattr(fc, "_current_stream", lambda: 0)
    monkeypatch.setattr(fc, "load", lambda: Library())
    return Past


BF, I4, F4 = ((4, 64), "bfloat16"), ((4,), "int32"), ((4,), "float32")
LISTS = dict(top_index=((4, 8), "int32"), top_logprob=((4, 8), "float32"))


@pytest.mark.parametrize("logits,others,say", [
    (((4, 64), "float16"), dict(lse=F4), "logits must be torch.bfloat16"),
    (((4, 64), "bfloat16", -1), dict(lse=F4), "logits must be on the device"),
    (((4, 64), "bfloat16", 1), dict(lse=F4), "not the current one"),
    (((4, 64), "bfloat16", 0, (1, 4)), dict(lse=F4), "unit column stride"),
    (BF, dict(lse=((4,), "float32", 1)), "lse must be on the logits' device 0"),
    (BF, dict(lse=((4,), "float32", -1)), "lse must be on the logits' device 0"),
    (BF, dict(lse=((4,), "float64")), "lse must be torch.float32"),
    (BF, dict(lse=((5,), "float32")), "lse must be"),
    (BF, dict(lse=((4,), "float32", 0, (2,))), "lse must be contiguous"),
    (BF, dict(tokens=((4,), "int64"), logprob=F4), "tokens must be torch.int32"),
    (BF, dict(tokens=I4, logprob=F4, keep=((4,), "bool")), "keep must be torch.uint8"),
    (BF, dict(top_index=((4, 8), "int64")), "top_index must be torch.int32"),
    (BF, dict(LISTS, top_logprob=((4, 7), "float32")), "top_logprob must be"),
    (BF, dict(LISTS, top_logprob=((4, 8), "float32", 0, (16, 1))), "same row stride"),
    (BF, dict(LISTS, lse=F4), None),
    (((1, 50257), "bfloat16", 0, (3, 1)), dict(lse=((1,), "float32")), None),
])
def test_binding_logprobs(fc, on_device_0, logits, others, say):
    args = {name: At(*v) for name, v in others.items()}
    with pytest.raises(ValueError if say else on_device_0, match=say):
        fc.axonn_token_logprobs(At(*logits), **args)


@pytest.mark.parametrize("others,say", [
    (dict(dlogits=((4, 64), "float32")), "dlogits must be torch.bfloat16"),
    (dict(dlogits=((4, 60), "bfloat16")), "dlogits must be"),
    (dict(lse=((4,), "bfloat16")), "lse must be torch.float32"),
    (dict(dlogprob=((3,), "float32")), "dlogprob must be"),
    (dict(dentropy=((4,), "float32", 1)), "dentropy must be on"),
    ({}, None),
])
def test_binding_backward(fc, on_device_0, others, say):
    args = {name: At(*v) for name, v in {**dict(lse=F4, dlogits=BF, tokens=I4, dlogprob=F4), **others}.items()}
    with pytest.raises(ValueError if say else on_device_0, match=say):
        fc.axonn_token_logprobs_bwd(At(*BF), **args)


@pytest.mark.parametrize("others,say", [
    (dict(top_logit=((4, 7), "float32")), "top_logit must be"),
    (dict(top_index=((4, 8), "int64")), "top_index must be torch.int32"),
    (dict(kept=((1,), "int64")), "kept must be torch.int32"),
    (dict(loss=((), "float32")), "loss must be"),
    (dict(dlogits=((4, 64), "bfloat16", 0, (1, 4))), "unit column stride"),
    ({}, None),
])
def test_binding_distill(fc, on_device_0, others, say):
    base = dict(top_index=((4, 8), "int32"), top_logit=((4, 8), "float32"), token_loss=F4, loss=((1,), "float32"),
                kept=((1,), "int32"), dlogits=BF)
    args = {name: At(*v) for name, v in {**base, **others}.items()}
    with pytest.raises(ValueError if say else on_device_0, match=say):
        fc.axonn_distill(At(*BF), **args)


# ------------------------------------------------------------------ lse in parts
def test_policy_gradient_against_differences_and_the_way_back():
    """The gradient from the logits alone: by differences, as the way back from
    64-bit lse and H, and for a row of any size."""
    rng = np.random.default_rng(6)
    tau = 0.6
    x = rng.normal(size=(4, 6))
    x[2, 1] = -np.inf
    tokens, g, h = np.array([2, -1, 5, 0]), rng.normal(size=4), rng.normal(size=4)
    f = vo.token_logprobs(x, tokens, None, tau)
    d = vo.policy_gradient(x, tokens, g, h, tau)
    assert np.allclose(d, vo.token_logprobs_bwd(x, f["lse"], tokens, g, f["entropy"], h, None, tau), rtol=0, atol=1e-14)
    step = 1e-5
    for at in np.ndindex(*x.shape):
        sides = []
        for s in (step, -step):
            y = x.copy()
            y[at] += s
            r = vo.token_logprobs(y, tokens, None, tau)
            sides.append((g * r["logprob"] + h * r["entropy"]).sum())
        assert abs((sides[0] - sides[1]) / (2 * step) - d[at]) < 1e-8  # step^2 f'''/6, and 1e-16 / step
    low = np.full((2, 5), -3.3895313892515355e38)
    low[1] = -np.inf
    d = vo.policy_gradient(low, np.array([1, 1]), np.ones(2), np.ones(2))
    assert np.allclose(d[0], np.array([-0.2, 0.8, -0.2, -0.2, -0.2])) and (d[1] == 0).all()


@pytest.mark.parametrize("fn,base,change", [
    ("axonn_token_logprobs", LOG, dict(flags=0x800)),                       # in parts, without lse
    ("axonn_token_logprobs_bwd", BWD, dict(flags=0x800, lse=0)),
    ("axonn_distill", DIS, dict(flags=0x800)),                              # has no lse
    ("axonn_token_logprobs", LOG, dict(flags=0x1800, lse=FAKE)),
])
def test_refusals_of_lse_in_parts(fc, fn, base, change):
    assert fc.LSE_PARTS == 0x800
    refuse(fc, fn, base, change, 1)


@pytest.mark.parametrize("lse,flags,say", [
    (((4,), "float32"), 0, None), (((4, 2), "float32"), 0x800, None),
    (((4, 3), "float32"), 0, "lse must be"), (((4, 1), "float32"), 0, "lse must be"), (((2, 2), "float32"), 0, "lse must be"),
    (((4, 2), "float64"), 0, "lse must be torch.float32"), (((4, 2), "float32", 0, (1, 4)), 0, "lse must be contiguous"),
    (((4, 2), "float32", 1), 0, "lse must be on the logits' device 0"),
])
def test_binding_of_lse_in_parts(fc, on_device_0, monkeypatch, lse, flags, say):
    """[T x 2] sets the flag, forward and backward."""
    got = []

    class Library:
        def __getattr__(self, name):
            def call(packed, stream):
                layout = fc._TOKEN_LOGPROBS if name == "axonn_token_logprobs" else fc._TOKEN_LOGPROBS_BWD
                got.append(layout.unpack(packed)[7])
                return 0
            return call
    monkeypatch.setattr(fc, "load", lambda: Library())
    calls = (lambda: fc.axonn_token_logprobs(At(*BF), lse=At(*lse)),
             lambda: fc.axonn_token_logprobs_bwd(At(*BF), At(*lse), At(*BF), tokens=At(*I4), dlogprob=At(*F4)))
    for call in calls:
        if say:
            with pytest.raises(ValueError, match=say):
                call()
        else:
            call()
    assert got == ([] if say else [flags, flags])


# ------------------------------------------------------------------ a student without a word left
def test_distill_where_the_student_has_no_probability():
    """The loss is infinite where q > 0 at p = 0, and the gradient p - q all the
    same: -q in a row of -inf alone, the other rows as they are without it."""
    rng = np.random.default_rng(7)
    x, t, tau = rng.normal(size=(3, 7)), rng.normal(size=(3, 3)), 1.5
    at = np.array([[0, 2, 4], [1, 3, 3], [6, 5, 0]])
    x[1] = -np.inf
    x[2, 6] = -np.inf
    r = vo.distill(x, at, t, None, tau, 2.0)
    q = np.exp(vo.log_softmax(t, tau))
    assert r["n"] == 3 and np.isfinite(r["token_loss"][0]) and (r["token_loss"][1:] == np.inf).all()
    want = np.zeros((3, 7))
    want[1, 1], want[1, 3] = -q[1, 0], -q[1, 1] - q[1, 2]
    want[2] = np.exp(vo.log_softmax(x[2:], tau))[0]
    want[2, at[2]] -= q[2]
    assert np.allclose(r["dlogits"][1:], want[1:] * 2.0 * tau / 3, rtol=1e-13, atol=0)
    alone = vo.distill(x[:1], at[:1], t[:1], None, tau, 2.0)
    assert np.allclose(r["dlogits"][0], alone["dlogits"][0] / 3, rtol=1e-13)
