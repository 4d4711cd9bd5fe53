"""The linear cross-entropy against its 64-bit form.

Bounds (derived).  A logit is a bf16 product accumulated in fp32: off by at
most e_z = (K/16 + 2) 2^-23 |X|.|W|.  The logsumexp and the label's logit are
each off by at most the row's largest e_z, plus 2^-21 of the logsumexp's
magnitude and 2^-20 for the exponentials' and the logarithm's own error; the
mean's bound is the mean of the rows'.  An entry of P is then relatively off
by twice that, by 2^-12 for a logit kept in 16 bits (half a step of 2^-11 in
the exponent, times ln 2; entries under 2^-32 of a group's maximum are 0) and
by its rounding to bf16 (half an ulp: 2^-8 of 8 significant bits), the label's
by the same of max(p, 1 - p) <= 1; dX and dW sum |P||W| and |X||P| of it,
accumulate in fp32 and round once.
"""
import numpy as np
import pytest

from oracle import epilogue as ep

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free_choice(cuda_lib):
    cuda_lib.axonn_set_kernel_config(-1)
    yield
    cuda_lib.axonn_set_kernel_config(-1)


def bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).to(torch.float64).numpy()


def dev(a, dtype, pad=8):
    import torch
    rows, cols = a.shape
    full = torch.full((rows, (cols + 7) // 8 * 8 + pad), float("nan"), dtype=dtype, device="cuda")
    full[:, :cols] = torch.from_numpy(a).to("cuda").to(dtype)
    return full[:, :cols]


def host(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def run(fc, X, W, labels, keep=None, tied=False, grad=True, dw="bf16", piece=0, scale=1.0, old=None):
    import torch
    T, K = X.shape
    V = W.shape[1]
    flags = (fc.B_T if tied else 0) | {"bf16": 0, "f32": fc.OUT_F32, "add": fc.ACCUM_F32}[dw]
    Wd = dev(W.T.copy() if tied else W, torch.bfloat16)
    o = {"token_loss": torch.full((T,), float("nan"), device="cuda"),
         "lse": torch.full((T,), float("nan"), device="cuda"),
         "loss": torch.full((1,), float("nan"), device="cuda"),
         "kept": torch.full((1,), -7, device="cuda", dtype=torch.int32)}
    if grad:
        o["dX"] = dev(np.full((T, K), 7.0), torch.bfloat16)
        kind = torch.bfloat16 if dw == "bf16" else torch.float32
        start = old if old is not None else np.full((K, V), 7.0)
        o["dW"] = dev(start.T.copy() if tied else start, kind)
    n = fc.axonn_linear_ce_workspace_size(T, K, V, flags, grad, piece)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")  # NaN in every format
    fc.axonn_linear_ce(dev(X, torch.bfloat16), Wd, torch.from_numpy(labels.astype(np.int32)).cuda(),
                       o["token_loss"], o["loss"], o["kept"], ws,
                       keep=None if keep is None else torch.from_numpy(keep.astype(np.uint8)).cuda(),
                       lse=o["lse"], dX=o.get("dX"), dW=o.get("dW"), grad_scale=scale, flags=flags)
    fc.axonn_sync_status()
    if grad:
        for t in (o["dX"], o["dW"]):
            assert bool(torch.isnan(t._base[:, t.shape[1]:].float()).all())  # the padding is untouched
    got = {k: host(v) for k, v in o.items()}
    if grad and tied:
        got["dW"] = got["dW"].T
    return got


def check(got, X, W, labels, keep=None, scale=1.0, dw="bf16", old=0.0):
    K = X.shape[1]
    r = ep.linear_ce(X, W, labels, keep, scale)
    c = r["counted"]
    assert got["kept"][0] == r["n"]
    assert (got["token_loss"][~c] == 0).all() and (got["lse"][~c] == 0).all()
    Xc = X[c]
    ez = (K / 16 + 2) * 2.0**-23 * (np.abs(Xc) @ np.abs(W))
    row = 2 * ez.max(axis=1, initial=0.0) + 2.0**-21 * np.abs(r["lse"][c]) + 2.0**-20
    assert (np.abs(got["lse"] - r["lse"])[c] <= row).all()
    assert (np.abs(got["token_loss"] - r["token_loss"])[c] <= row).all()
    n = max(r["n"], 1)
    assert abs(got["loss"][0] - r["loss"]) <= row.sum() / n + 2.0**-20 * abs(r["loss"])
    if "dX" not in got:
        return
    P = np.abs(r["P"])
    eP = P * (2.0**-8 + 2.0**-12 + 2 * row[:, None]) + 2.0**-32 * abs(scale) / n
    y = labels[c]
    at = (np.arange(len(y)), y)
    eP[at] += 2 * row * abs(scale) / n  # the label's entry: p - 1 has p's absolute error
    bX = np.zeros_like(X)
    bX[c] = eP @ np.abs(W).T + (W.shape[1] / 16 + 2) * 2.0**-23 * (P @ np.abs(W).T)
    bW = np.abs(Xc).T @ eP + (len(y) / 16 + 2) * 2.0**-23 * (np.abs(Xc).T @ P)
    assert (got["dX"][~c] == 0).all()
    assert (np.abs(got["dX"] - r["dX"]) <= bX + 2.0**-8 * np.abs(r["dX"]) + 1e-30).all()
    want = r["dW"] + old
    unit = 2.0**-8 if dw == "bf16" else 2.0**-22
    assert (np.abs(got["dW"] - want) <= bW + unit * (np.abs(want) + np.abs(old)) + 1e-30).all()


def case(T, K, V, seed=1, spread=1.0):
    rng = np.random.default_rng(seed)
    X = bf16(rng.normal(size=(T, K)))
    W = bf16(rng.normal(size=(K, V)) * spread / np.sqrt(K))
    return X, W, rng.integers(0, V, size=T), rng


SIZES = [(1, 8, 1), (1, 64, 1000), (2, 72, 257), (33, 130, 300), (130, 64, 1003), (300, 200, 2000), (257, 40, 4097)]


@pytest.mark.parametrize("config", [2, 0, 6, 7])
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_against_64_bits(cuda_lib, size, tied, config):
    X, W, labels, rng = case(*size)
    cuda_lib.axonn_set_kernel_config(config)
    check(run(cuda_lib, X, W, labels, tied=tied), X, W, labels)


@pytest.mark.parametrize("piece", [1, 512, 1024])
@pytest.mark.parametrize("tied", [False, True])
def test_in_pieces(cuda_lib, piece, tied):
    """Pieces of 256, 512 and 1024 columns of a 1990-token vocabulary: the
    last one short, and all but one computed again."""
    X, W, labels, rng = case(200, 72, 1990, seed=4)
    labels[::7] = -1
    got = run(cuda_lib, X, W, labels, tied=tied, piece=piece)
    check(got, X, W, labels)
    loss = run(cuda_lib, X, W, labels, tied=tied, grad=False)
    check(loss, X, W, labels)


@pytest.mark.parametrize("dw", ["f32", "add"])
@pytest.mark.parametrize("piece", [0, 256])
def test_fp32_weight_gradient(cuda_lib, dw, piece):
    X, W, labels, rng = case(150, 64, 700, seed=6)
    old = rng.normal(size=W.shape).astype(np.float32).astype(np.float64)
    got = run(cuda_lib, X, W, labels, dw=dw, piece=piece, scale=64.0, old=old)
    check(got, X, W, labels, scale=64.0, dw=dw, old=old if dw == "add" else 0.0)


@pytest.mark.parametrize("which", ["none", "all", "one", "half", "keep"])
@pytest.mark.parametrize("piece", [0, 256])
def test_masks(cuda_lib, which, piece):
    """Rows that do not count hold NaN and infinities; nothing of them is
    seen, and a mask may leave nothing at all."""
    X, W, labels, rng = case(130, 72, 600, seed=8)
    keep = None
    if which == "none":
        labels[:] = 600
    elif which == "one":
        labels[np.arange(130) != 77] = -100
    elif which == "half":
        labels[rng.random(130) < 0.5] = -1
    elif which == "keep":
        keep = (rng.random(130) < 0.5).astype(np.uint8) * 3
    counted = (labels >= 0) & (labels < 600) & (keep != 0 if keep is not None else True)
    dirty = X.copy()
    dirty[~counted] = np.where(rng.random((int((~counted).sum()), 72)) < 0.5, np.nan, np.inf)
    got = run(cuda_lib, dirty, W, labels, keep, piece=piece)
    check(got, X, W, labels, keep)


def test_confident_rows(cuda_lib):
    """Logits of +-60: a label with probability near 1 has a small gradient
    of its own, the others underflow to 0, and a label far below the maximum
    has a large loss."""
    T, K, V = 64, 32, 900
    rng = np.random.default_rng(2)
    X, W = bf16(np.eye(T, K) * 60 + np.eye(T, K, -32) * 60), bf16(rng.choice([-1.0, 1.0], size=(K, V)) * 0.5)
    labels = rng.integers(0, V, size=T)
    for t in range(32):
        W[t % K, labels[t]] = 1.0   # the only largest logit of rows t and t + 32
    check(run(cuda_lib, X, W, labels), X, W, labels)
    check(run(cuda_lib, X, W, labels, piece=256), X, W, labels)


def test_infinite_and_nan_logits(cuda_lib):
    """A column of -inf logits has probability 0; a row with a NaN has a NaN
    loss, and no other row does."""
    import torch
    X, W, labels, rng = case(40, 16, 300, seed=12)
    X = np.abs(X) + 0.5
    X = bf16(X)
    Wi = W.copy()
    Wi[0, 5] = -np.inf
    labels[labels == 5] = 6
    got = run(cuda_lib, X, Wi, labels)
    Wf = W.copy()
    Wf[:, 5] = bf16(np.full(16, -1e30))   # as good as -inf in 64 bits
    r = ep.linear_ce(X, Wf, labels)
    assert np.abs(got["token_loss"] - r["token_loss"]).max() < 1e-4
    X[7, 3] = np.nan
    got = run(cuda_lib, X, W, labels, grad=False)
    assert np.isnan(got["token_loss"][7]) and np.isfinite(np.delete(got["token_loss"], 7)).all()


def test_empty(cuda_lib):
    """No positions: loss 0, nothing counted, a zero weight gradient (an
    unchanged one where it accumulates)."""
    X, W, labels, _ = case(0, 16, 50)
    got = run(cuda_lib, X, W, labels)
    assert got["loss"][0] == 0 and got["kept"][0] == 0 and (got["dW"] == 0).all()
    got = run(cuda_lib, X, W, labels, dw="add")
    assert (got["dW"] == 7).all()


def test_loss_does_not_depend_on_the_workspace(cuda_lib):
    """Same statistics whatever is kept: the loss is the same number, and it
    is the same on every run."""
    X, W, labels, _ = case(300, 128, 3000 // 2, seed=5)
    a, b, c = (run(cuda_lib, X, W, labels, grad=g, piece=p) for g, p in ((True, 0), (True, 0), (False, 0)))
    assert np.array_equal(a["token_loss"], b["token_loss"]) and np.array_equal(a["token_loss"], c["token_loss"])
    assert np.array_equal(a["dX"], b["dX"]) and np.array_equal(a["dW"], b["dW"])


def test_expired_wait_is_reported(cuda_lib):
    """Operand loads withheld: the bounded waits expire, the status says so,
    and the next call is right."""
    fc = cuda_lib
    X, W, labels, _ = case(40, 64, 300)
    fc.axonn_set_wait_timeout_ns(2_000_000)
    fc.axonn_debug_set_inject(1)
    try:
        with pytest.raises(fc.AxonnError) as e:
            run(fc, X, W, labels, grad=False)
        assert e.value.status == fc.ERR_TIMEOUT
    finally:
        fc.axonn_debug_set_inject(0)
        fc.axonn_set_wait_timeout_ns(4_000_000_000)
    check(run(fc, X, W, labels), X, W, labels)


@pytest.mark.parametrize("n", [31, 32, 33, 64, 65, 96, 128, 129])
@pytest.mark.parametrize("piece", [0, 256])
def test_counted_rows_at_the_edges_of_a_tile(cuda_lib, n, piece):
    """The weight gradient's reduction runs in steps of 64 packed rows, an
    epilogue warp owns 32: whatever lies past the last row adds nothing.  The
    workspace starts as NaN."""
    X, W, labels, rng = case(200, 72, 700, seed=20 + n)
    keep = np.zeros(200, dtype=np.uint8)
    keep[rng.permutation(200)[:n]] = 1
    for config in (6, 2, 0, 7):
        cuda_lib.axonn_set_kernel_config(config)
        check(run(cuda_lib, X, W, labels, keep, piece=piece), X, W, labels, keep)


def test_no_features(cuda_lib):
    """K = 0: every logit is 0 and the loss is ln V."""
    X, W = np.zeros((20, 0)), np.zeros((0, 300))
    got = run(cuda_lib, X, W, np.arange(20), grad=False)
    assert np.abs(got["token_loss"] - np.log(300.0)).max() < 1e-5 and got["kept"][0] == 20


def test_offsets_past_32_bits(cuda_lib):
    """A piece of more than 2^31 entries: the losses and dX of the last rows,
    and dW of the last columns, against 64 bits."""
    fc = cuda_lib
    import torch
    T, K, V, tail = 16800, 64, 128256, 40
    assert T * V > 2**31
    g = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn((T, K), device="cuda", generator=g).to(torch.bfloat16)
    W = torch.randn((K, V), device="cuda", generator=g).mul_(0.1).to(torch.bfloat16)
    labels = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    tl, loss = torch.empty(T, device="cuda"), torch.empty(1, device="cuda")
    kept = torch.empty(1, device="cuda", dtype=torch.int32)
    ws = torch.empty(fc.axonn_linear_ce_workspace_size(T, K, V, piece=V), device="cuda", dtype=torch.uint8)
    fc.axonn_linear_ce(X, W, labels, tl, loss, kept, ws, dX=dX, dW=dW)
    fc.axonn_sync_status()
    z = X[-tail:].double() @ W.double()
    logp = torch.log_softmax(z, dim=1)
    y = labels[-tail:].long()
    at = torch.arange(tail, device="cuda")
    assert float((tl[-tail:].double() + logp[at, y]).abs().max()) < 1e-4
    P = logp.exp()
    P[at, y] -= 1
    ref = P @ W.double().T / T
    assert float((dX[-tail:].double() - ref).norm() / ref.norm()) < 2 * 2.0**-8
    # dW's last columns: every row's probabilities there
    lse = torch.cat([torch.logsumexp(X[i:i + 2100].double() @ W.double(), dim=1) for i in range(0, T, 2100)])
    cols = W[:, -24:].double()
    P = torch.exp(X.double() @ cols - lse[:, None])
    hit = labels.long()[:, None] == torch.arange(V - 24, V, device="cuda")
    ref = X.double().T @ (P - hit.double()) / T
    assert float((dW[:, -24:].double() - ref).norm() / ref.norm()) < 2 * 2.0**-8


@pytest.mark.parametrize("piece", [0, 256])
@pytest.mark.parametrize("where", ["row", "column"])
def test_nan_reaches_every_entry_it_should(cuda_lib, where, piece):
    """Logits so far apart that most probabilities are 0: a NaN in a counted
    row or in a column of W still shows in all the gradients that contain it,
    and in no other."""
    rng = np.random.default_rng(11)
    T, K, V = 40, 64, 700
    X, W = bf16(20 * rng.standard_normal((T, K))), bf16(rng.standard_normal((K, V)))
    labels = rng.integers(0, V, T)
    labels[5] = -1
    if where == "row":
        X[7, 3] = np.nan
        X[5] = np.nan  # does not count
    else:
        W[9, 17] = np.nan
    got = run(cuda_lib, X, W, labels, piece=piece)
    counted = labels >= 0
    hit = counted & (np.arange(T) == 7) if where == "row" else counted
    assert (np.isnan(got["token_loss"]) == hit).all() and np.isnan(got["loss"]).all()
    assert (np.isnan(got["dX"]) == hit[:, None]).all() and (got["dX"][5] == 0).all()
    assert np.isnan(got["dW"]).all()


# Above 256 features the last piece of the vocabulary is kept as distances
# (above 512 where it is larger than L2) instead of being computed again.
KEPT = [(1, 264, 1000), (33, 272, 300), (130, 520, 1003), (300, 300, 2000), (257, 264, 4097)]


@pytest.mark.parametrize("config", [2, 0, 6, 7])
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("size", KEPT)
def test_kept_piece_against_64_bits(cuda_lib, size, tied, config):
    X, W, labels, rng = case(*size, seed=31)
    cuda_lib.axonn_set_kernel_config(config)
    check(run(cuda_lib, X, W, labels, tied=tied), X, W, labels)


@pytest.mark.parametrize("K", [256, 257, 264])
@pytest.mark.parametrize("n", [0, 1, 31, 64, 65, 129])
def test_kept_piece_and_counted_rows(cuda_lib, K, n):
    """Both sides of the number of features up to which the piece is computed
    again, with a vocabulary that ends inside 16 bytes; the other rows hold
    NaN."""
    T, V = 150, 701
    X, W, labels, rng = case(T, K, V, seed=40 + n)
    keep = np.zeros(T, dtype=np.uint8)
    keep[rng.permutation(T)[:n]] = 1
    dirty = X.copy()
    dirty[keep == 0] = np.nan
    for piece in (0, 256):
        check(run(cuda_lib, dirty, W, labels, keep, piece=piece), X, W, labels, keep)


@pytest.mark.parametrize("dw", ["f32", "add"])
@pytest.mark.parametrize("piece", [0, 256])
def test_kept_piece_fp32_weight_gradient(cuda_lib, dw, piece):
    X, W, labels, rng = case(150, 264, 700, seed=36)
    old = rng.normal(size=W.shape).astype(np.float32).astype(np.float64)
    got = run(cuda_lib, X, W, labels, dw=dw, piece=piece, scale=64.0, old=old)
    check(got, X, W, labels, scale=64.0, dw=dw, old=old if dw == "add" else 0.0)


@pytest.mark.parametrize("piece", [0, 256])
def test_kept_piece_confident_rows(cuda_lib, piece):
    """Logits so far apart that most probabilities are 0 and a label's is
    near 1, or near 0."""
    T, K, V = 64, 264, 900
    X, W, labels, rng = case(T, K, V, seed=33, spread=20.0)
    labels[::2] = (X @ W).argmax(axis=1)[::2]
    check(run(cuda_lib, X, W, labels, piece=piece), X, W, labels)


@pytest.mark.parametrize("where", ["row", "column"])
def test_kept_piece_nan(cuda_lib, where):
    """As test_nan_reaches_every_entry_it_should, with a kept piece."""
    T, K, V = 40, 264, 700
    X, W, labels, rng = case(T, K, V, seed=37, spread=20.0)
    labels[5] = -1
    if where == "row":
        X[7, 3] = np.nan
        X[5] = np.nan  # does not count
    else:
        W[9, 17] = np.nan
    got = run(cuda_lib, X, W, labels)
    counted = labels >= 0
    hit = counted & (np.arange(T) == 7) if where == "row" else counted
    assert (np.isnan(got["token_loss"]) == hit).all() and np.isnan(got["loss"]).all()
    assert (np.isnan(got["dX"]) == hit[:, None]).all() and (got["dX"][5] == 0).all()
    assert np.isnan(got["dW"]).all()


def test_kept_piece_offsets_past_32_bits(cuda_lib):
    """A kept piece of more than 2^31 entries: dX of the last rows, and dW of
    the last columns, against 64 bits."""
    fc = cuda_lib
    import torch
    T, K, V, tail = 16800, 520, 128256, 40
    assert T * V > 2**31
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn((T, K), device="cuda", generator=g).to(torch.bfloat16)
    W = torch.randn((K, V), device="cuda", generator=g).mul_(0.04).to(torch.bfloat16)
    labels = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    tl, loss = torch.empty(T, device="cuda"), torch.empty(1, device="cuda")
    kept = torch.empty(1, device="cuda", dtype=torch.int32)
    ws = torch.empty(fc.axonn_linear_ce_workspace_size(T, K, V, piece=V), device="cuda", dtype=torch.uint8)
    fc.axonn_linear_ce(X, W, labels, tl, loss, kept, ws, dX=dX, dW=dW)
    fc.axonn_sync_status()
    z = X[-tail:].double() @ W.double()
    logp = torch.log_softmax(z, dim=1)
    y = labels[-tail:].long()
    at = torch.arange(tail, device="cuda")
    assert float((tl[-tail:].double() + logp[at, y]).abs().max()) < 1e-4
    P = logp.exp()
    P[at, y] -= 1
    ref = P @ W.double().T / T
    assert float((dX[-tail:].double() - ref).norm() / ref.norm()) < 2 * 2.0**-8
    cols = W[:, -24:].float()
    lse = torch.cat([torch.logsumexp(X[i:i + 2100].float() @ W.float(), dim=1) for i in range(0, T, 2100)])
    P = torch.exp(X.double() @ cols.double() - lse.double()[:, None])
    hit = labels.long()[:, None] == torch.arange(V - 24, V, device="cuda")
    ref = X.double().T @ (P - hit.double()) / T
    assert float((dW[:, -24:].double() - ref).norm() / ref.norm()) < 2 * 2.0**-8


@pytest.mark.parametrize("K", [72, 264, 520])
@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 65, 149])
@pytest.mark.parametrize("V", [4097, 20000])
def test_parts_of_dx_follow_the_counted_rows(cuda_lib, V, n, K):
    """dX as fp32 parts of a reduction over a long vocabulary: how many, and
    how far apart, follows on the device from the rows that count.  The other
    rows hold NaN, and so does the workspace at the start."""
    T = 150
    X, W, labels, rng = case(T, K, V, seed=50 + n)
    size = lambda v: (cuda_lib.axonn_linear_ce_workspace_size(T, K, v)  # noqa: E731
                      - cuda_lib.axonn_linear_ce_workspace_size(T, K, v, grad=False))
    assert size(V) >= 2 * T * V + 2 * 4 * T * K  # at least two parts
    keep = np.zeros(T, dtype=np.uint8)
    keep[rng.permutation(T)[:n]] = 1
    dirty = X.copy()
    dirty[keep == 0] = np.nan
    check(run(cuda_lib, dirty, W, labels, keep, tied=n % 2 == 1), X, W, labels, keep)


@pytest.mark.parametrize("K", [72, 264])
@pytest.mark.parametrize("size", [(1100, 14000), (1100, 11000), (600, 14003)])
@pytest.mark.parametrize("config", [6, 2, 0, 7])
def test_tiles_in_rounds(cuda_lib, config, size, K):
    """More tiles than run at once: statistics, probabilities (computed again,
    and from the kept piece) and the two gradients, with a last round that
    fills less and more than half of the units."""
    T, V = size
    X, W, labels, rng = case(T, K, V, seed=60)
    labels[::9] = -100
    cuda_lib.axonn_set_kernel_config(config)
    check(run(cuda_lib, X, W, labels), X, W, labels)


@pytest.mark.parametrize("piece", [0, 512])
@pytest.mark.parametrize("tied", [False, True])
def test_one_gradient_alone(cuda_lib, tied, piece):
    """dX without dW and dW without dX are the same numbers as together."""
    import torch
    fc = cuda_lib
    T, K, V = 130, 264, 5003
    X, W, labels, rng = case(T, K, V, seed=70)
    labels[::5] = -1
    Xd, Wd = dev(X, torch.bfloat16), dev(W.T.copy() if tied else W, torch.bfloat16)
    y = torch.from_numpy(labels.astype(np.int32)).cuda()
    flags = fc.B_T if tied else 0
    ws = torch.full((fc.axonn_linear_ce_workspace_size(T, K, V, flags, True, piece),), 255, dtype=torch.uint8,
                    device="cuda")
    got = []
    for want in ("both", "dX", "dW"):
        dX, dW = (torch.zeros_like(t) if want in ("both", n) else None for n, t in (("dX", Xd), ("dW", Wd)))
        if dX is not None:
            dX = dev(np.full((T, K), 7.0), torch.bfloat16)
        if dW is not None:
            dW = dev(np.full(Wd.shape, 7.0), torch.bfloat16)
        out = [torch.empty(T, device="cuda"), torch.empty(1, device="cuda"),
               torch.empty(1, device="cuda", dtype=torch.int32)]
        fc.axonn_linear_ce(Xd, Wd, y, *out, ws, dX=dX, dW=dW, flags=flags)
        fc.axonn_sync_status()
        got.append((out, dX, dW))
    for out, dX, dW in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out, got[0][0]))
        assert dX is None or torch.equal(dX, got[0][1])
        assert dW is None or torch.equal(dW, got[0][2])


def test_two_streams_at_once(cuda_lib):
    """A loss with gradients and a layer with its epilogue on two streams,
    again and again: each as when it runs alone."""
    import torch
    fc = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(9)
    T, K, V, N = 700, 264, 9000, 1040

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)

    X, W, W1, Z = rand(T, K), rand(K, V).mul_(0.05), rand(K, N).mul_(0.05), rand(T, N)
    labels = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    ws = torch.empty(fc.axonn_linear_ce_workspace_size(T, K, V), dtype=torch.uint8, device="cuda")
    epi_ws = torch.empty(fc.axonn_epi_workspace_size(T, K), dtype=torch.uint8, device="cuda")
    rng = torch.tensor([5, 6], device="cuda")

    def loss(o, s):
        fc.axonn_linear_ce(X, W, labels, o[0], o[1], o[2], ws, dX=o[3], dW=o[4], stream=s)

    def layer(o, s):
        fc.axonn_fc_fwd_epi(X, W1, o[0], fc.Shape(T, K, N), act="gelu", residual=Z, p=0.2, rng=rng, stream=s)
        fc.axonn_fc_dgrad_epi(o[0], W1, o[1], fc.Shape(T, K, N), pre=X, act="silu", dbias=o[2], ws=epi_ws, stream=s)
        fc.axonn_fc_fwd_epi(X[:2], W1, o[3], fc.Shape(2, K, N), act="silu", stream=s)

    def outputs():
        e = lambda *shape, t=torch.float32: torch.empty(shape, device="cuda", dtype=t)  # noqa: E731
        b = torch.bfloat16
        return ([e(T), e(1), e(1, t=torch.int32), e(T, K, t=b), e(K, V, t=b)],
                [e(T, N, t=b), e(T, K, t=b), e(K), e(2, N, t=b)])

    alone, both = outputs(), outputs()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    loss(alone[0], None)
    layer(alone[1], None)
    torch.cuda.synchronize()
    for _ in range(20):
        loss(both[0], streams[0])
        for _ in range(4):
            layer(both[1], streams[1])
    for s in streams:
        fc.axonn_sync_status(s)
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
