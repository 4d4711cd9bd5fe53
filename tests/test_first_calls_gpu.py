"""What a process pays at its first calls, each script in a process of its
own."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = """
import json, sys, time
sys.path.insert(0, sys.argv[1])
import torch
import pmm_fc_layer_gb300 as fc
fc.load()
x = torch.eye(64, device="cuda", dtype=torch.bfloat16)
y = torch.empty_like(x)
shape = fc.Shape(64, 64, 64)
b = torch.ones(64, device="cuda")
torch.cuda.synchronize()
def ms(f):
    t = time.perf_counter()
    f()
    return (time.perf_counter() - t) * 1e3
"""


def run(script):
    out = subprocess.run([sys.executable, "-c", PRELUDE + script, ROOT], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    return json.loads(out.stdout.strip().splitlines()[-1])


def test_plain_products_do_not_set_up_the_fused_ones(cuda_lib):
    """The fused kernels take longer to set up than all the others; that falls
    to the first call that needs them."""
    got = run("""
plain = ms(lambda: fc.axonn_fc_fwd(x, x, y, shape))
fused = ms(lambda: fc.axonn_fc_fwd_epi(x, x, y, shape, bias=b))
fc.axonn_sync_status()
print(json.dumps([plain, fused]))
""")
    assert got[0] < got[1], got


def test_first_fused_call_inside_a_capture(cuda_lib):
    """After a plain product, the first fused one may be a captured one."""
    got = run("""
fc.axonn_fc_fwd(x, x, y, shape)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fc.axonn_fc_fwd_epi(x, x, y, shape, bias=b)
y.zero_()
g.replay()
fc.axonn_sync_status()
print(json.dumps(bool(torch.equal(y.float(), torch.eye(64, device="cuda") + 1.0))))
""")
    assert got is True


def test_status_of_plain_products_waits_for_their_words_alone(cuda_lib):
    """Each group of kernels has a status word that is copied to the host; a
    process without fused products does not wait for theirs: four copies where
    the others make six."""
    got = run("""
def status_us():
    fc.axonn_sync_status()
    n = 200
    return min(ms(lambda: [fc.axonn_sync_status() for _ in range(n)]) for _ in range(5)) / n * 1e3
fc.axonn_fc_fwd(x, x, y, shape)
plain = status_us()
fc.axonn_fc_fwd_epi(x, x, y, shape, bias=b)
print(json.dumps([plain, status_us()]))
""")
    assert got[0] < 0.75 * got[1], got
