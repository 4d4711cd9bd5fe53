"""Several host threads calling the C ABI at once, each on its own stream."""
import threading

import numpy as np
import pytest

import oracle
from fc_cases import host_bits, make_operand, operand_names, to_device

pytestmark = pytest.mark.gpu


def test_concurrent_calls_on_separate_streams(cuda_lib):
    import torch
    fc = cuda_lib
    cases = []
    for i, (op, (T, K, N)) in enumerate([("fwd", (300, 200, 520)), ("dgrad", (256, 384, 640)),
                                         ("wgrad", (512, 136, 264)), ("fwd", (1024, 512, 768))]):
        pn, qn = operand_names(op)
        P = make_operand(pn, T, K, N, False, seed=300 + i, kind="int")
        Q = make_operand(qn, T, K, N, False, seed=300 + i, kind="int")
        want = oracle.bf16_rne(oracle.fc(op, P, Q)[0])
        cases.append((op, T, K, N, to_device(P), to_device(Q), want))
    results, errors = {}, []

    def worker(idx):
        try:
            op, T, K, N, Pd, Qd, _ = cases[idx]
            s = torch.cuda.Stream()
            M, Nn = fc.out_shape(op, T, K, N)
            out = torch.empty((M, ((Nn + 7) // 8) * 8), dtype=torch.bfloat16, device="cuda")[:, :Nn]
            for _ in range(20):
                fc.call(op, Pd, Qd, out, fc.Shape(T, K, N), 0, None, stream=s)
            fc.axonn_sync_status(s)
            results[idx] = host_bits(out)
        except Exception as e:  # reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i, case in enumerate(cases):
        assert np.array_equal(results[i], case[-1]), i


def test_rows_of_different_reductions_from_several_threads(cuda_lib):
    """Products of two rows need shared memory by the length of their
    reduction; calls of different lengths at once, each on its own stream, are
    all taken.  The calls are short and made through the C interface, so that
    the threads spend their time inside it."""
    import ctypes

    import torch
    fc = cuda_lib
    N, calls = 64, 4000
    lib, epilogue = fc.load(), fc.Epilogue()
    g = torch.Generator(device="cuda").manual_seed(1)
    cases = []
    for K in (65536, 49152, 65536, 49152, 57344, 65536):
        X = torch.randn((2, K), device="cuda", generator=g).to(torch.bfloat16)
        W = torch.randn((K, N), device="cuda", generator=g).mul_(0.02).to(torch.bfloat16)
        cases.append((K, X, W, torch.empty((2, N), device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    refused = []
    start = threading.Barrier(len(cases))

    def worker(K, X, W, Y, s):
        shape = fc.Shape(2, K, N)
        args = (X.data_ptr(), W.data_ptr(), Y.data_ptr(), K, N, N, ctypes.byref(shape), fc.OUT_F32,
                ctypes.byref(epilogue), s.cuda_stream)
        start.wait()
        for _ in range(calls):
            st = lib.axonn_fc_fwd_epi(*args)
            if st != fc.OK:
                refused.append((K, st, lib.axonn_last_error()))

    threads = [threading.Thread(target=worker, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, (len(refused), refused[0])
    for K, X, W, Y, _ in cases:
        ref = X.double() @ W.double()
        # products of bf16 numbers are exact in fp32; K of them are added up
        assert bool(((Y.double() - ref).abs() <= K * 2.0**-24 * (X.double().abs() @ W.double().abs())).all())
