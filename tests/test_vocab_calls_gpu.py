"""The operators over rows of logits from several host threads at once, each
on its own stream, and as the first calls of a process."""
import json
import os
import subprocess
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Work:
    """A few rows with their lists, and what the operators leave for them."""

    def __init__(self, seed, T, V):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = dict(device="cuda", dtype=torch.bfloat16)
        self.X = torch.randn((T, V), device="cuda", generator=g).to(torch.bfloat16)
        self.index = torch.empty((T, 8), device="cuda", dtype=torch.int32)
        self.value, self.lse, self.token = torch.empty((T, 8), device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        self.loss, self.kept = torch.empty(1, device="cuda"), torch.empty(1, device="cuda", dtype=torch.int32)
        self.d, self.d2 = torch.empty((T, V), **bf), torch.empty((T, V), **bf)
        self.g = torch.randn(T, device="cuda", generator=g)

    def run(self, fc, stream=None):
        fc.axonn_token_logprobs(self.X, lse=self.lse, top_index=self.index, top_logprob=self.value, stream=stream)
        fc.axonn_token_logprobs_bwd(self.X, self.lse, self.d, tokens=self.index[:, 0].contiguous(), dlogprob=self.g,
                                    stream=stream)
        fc.axonn_distill(self.X, self.index, self.value, self.token, self.loss, self.kept, dlogits=self.d2,
                         temperature=2.0, stream=stream)

    def left(self):
        return [t.clone() for t in (self.index, self.value, self.lse, self.token, self.loss, self.kept, self.d, self.d2)]


def test_several_threads(cuda_lib):
    """The same results as alone, whatever runs beside: rows in shares, in a
    ring of buffers, short and long."""
    import torch
    fc = cuda_lib
    sizes = [(3, 40000), (310, 32768), (700, 2048), (40, 128256)]
    work = [Work(i, *s) for i, s in enumerate(sizes)]
    want = []
    for w in work:
        w.run(fc)
        torch.cuda.synchronize()
        want.append(w.left())
    errors = []

    def worker(w):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(15):
                    w.run(fc)
            fc.axonn_sync_status(stream)
        except Exception as e:  # reported below
            errors.append(repr(e))
    threads = [threading.Thread(target=worker, args=(w,)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for w, old in zip(work, want):
        assert all(torch.equal(a, b) for a, b in zip(w.left(), old))


@pytest.mark.parametrize("pdl", [0, 1])
def test_plain_and_dependent_launches_agree(cuda_lib, pdl):
    import torch
    fc = cuda_lib
    w = Work(7, 320, 30000)
    w.run(fc)
    torch.cuda.synchronize()
    want = w.left()
    try:
        fc.axonn_set_pdl(pdl)
        for _ in range(5):
            w.run(fc)
        fc.axonn_sync_status()
    finally:
        fc.axonn_set_pdl(1)
    assert all(torch.equal(a, b) for a, b in zip(w.left(), want))


def test_first_calls_inside_a_capture(cuda_lib):
    """A process's first calls may be captured ones."""
    script = """
import json, sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import pmm_fc_layer_gb300 as fc
from test_vocab_calls_gpu import Work
fc.load()
w = Work(3, 320, 30000)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    w.run(fc)
g.replay()
fc.axonn_sync_status()
got = w.left()
for t in (w.index, w.value, w.lse, w.token, w.loss, w.kept, w.d, w.d2):
    t.zero_()
w.run(fc)
fc.axonn_sync_status()
print(json.dumps(all(bool(torch.equal(a, b)) for a, b in zip(w.left(), got))))
"""
    out = subprocess.run([sys.executable, "-c", script, ROOT], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert json.loads(out.stdout.strip().splitlines()[-1]) is True
