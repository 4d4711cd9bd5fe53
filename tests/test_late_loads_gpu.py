"""Loads that land after the wait for them has run out: the call reports it, and
nothing that comes later is harmed."""
import numpy as np
import pytest

from oracle import goldfish as gf
from test_goldfish_gpu import _check, _problem, _run
from test_vocab_gpu import lists_of, logits_of, run_distill

pytestmark = pytest.mark.gpu


def late(fc, call):
    """The call with the first load of each CTA held back beyond the limit."""
    fc.axonn_set_wait_timeout_ns(20_000_000)
    fc.axonn_debug_set_inject(2)
    try:
        with pytest.raises(fc.AxonnError) as e:
            call()
        assert e.value.status == fc.ERR_TIMEOUT
    finally:
        fc.axonn_debug_set_inject(0)
        fc.axonn_set_wait_timeout_ns(4_000_000_000)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind,V", [("bf16", 33000), ("f32", 70007), ("bf16", 131076)])
def test_distill(cuda_lib, kind, V, in_place):
    """A CTA's last copies fit its buffers, so that its producer waits for nobody
    (three chunks a row), or do not."""
    fc, kinds, T = cuda_lib, 13, 310
    x, _, rng = logits_of(kinds, V, kind, seed=36)
    at, t = lists_of(x, 8, rng)
    pick = np.arange(T) % kinds
    args = (fc, x[pick], kind, at[pick], t[pick])
    want = run_distill(*args, in_place=in_place)
    for _ in range(2):
        late(fc, lambda: run_distill(*args, in_place=in_place))
        again = run_distill(*args, in_place=in_place)
        assert all(np.array_equal(want[n], again[n]) for n in want)


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("V", [20000, 128256])
def test_goldfish(cuda_lib, V, grad):
    """Two rows' copies fit the buffers, or one row's do not."""
    fc = cuda_lib
    ids, labels, logits = _problem(2, 200, V, 305)
    want = _run(fc, ids, labels, logits, 0, 13, grad=grad)
    few = (ids[:1, :40], labels[:1, :40], logits[:40])
    _check(_run(fc, *few, 0, 13, grad=grad), gf.goldfish_ce(few[2], *few[:2], 0, 13), V, few[2])
    for _ in range(2):
        late(fc, lambda: _run(fc, ids, labels, logits, 0, 13, grad=grad))
        again = _run(fc, ids, labels, logits, 0, 13, grad=grad)
        assert all(np.array_equal(want[n], again[n]) for n in want if want[n] is not None)
