"""The bounded waits of every 8-bit integer kernel and way of handing out work,
made to run out as in test_gpu_i8_timeout.py (2 ms limits, producers that arm
their barriers without a copy): each call returns, reports MPQ_ERR_TIMEOUT once
and leaves the context usable."""
import ctypes
import time

import pytest

import i8_shapes
from test_gpu_i8 import assert_close, product64, rand_i8, u
from test_gpu_i8_timeout import libs  # noqa: F401

pytestmark = pytest.mark.gpu

GROUPS = sorted({c[:4] for c in i8_shapes.cases()})


@pytest.mark.parametrize("op,part,kernel,columns", GROUPS)
def test_waits_run_out(libs, op, part, kernel, columns):
    import torch
    mpq, _lib, wt = libs
    r, P = ctypes.byref, lambda t: ctypes.c_void_p(t.data_ptr())
    s = _lib._stream()
    for case in i8_shapes.cases():
        if case[:4] != (op, part, kernel, columns):
            continue
        M, N, K = case[5:]
        assert i8_shapes.classes(mpq.i8_plan(op, M, N, K))[part] == (kernel, columns, case[4])
        x, wg, wu = rand_i8(mpq, M, K, 1), rand_i8(mpq, N, K, 2), rand_i8(mpq, N, K, 3)
        dh = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
        h = torch.empty(M, N, device="cuda")
        dg, du = torch.empty_like(dh), torch.empty_like(dh)
        dx = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
        ws = torch.zeros(getattr(wt, "mpq_i8_%s_workspace_size" % op)(M, N, K), dtype=torch.uint8, device="cuda")
        w = (P(ws), ws.numel(), s)
        call = {
            "linear": lambda: wt.mpq_i8_linear(r(x.c), r(wg.c), P(h), 0, N, *w),
            "gated": lambda: wt.mpq_i8_gated(r(x.c), r(wg.c), r(wu.c), 0, P(h), 0, N, *w),
            "linear_backward": lambda: wt.mpq_i8_linear_backward(r(wg.c), P(dh), M, N, P(dx), K, *w),
            "gated_backward": lambda: wt.mpq_i8_gated_backward(r(x.c), r(wg.c), r(wu.c), 0, P(dh), N, P(dg), P(du), N,
                                                               P(dx), K, *w),
        }[op]
        t0 = time.perf_counter()
        assert call() == 0, case
        assert _lib.STATUS[wt.mpq_check(P(ws), s)] == "MPQ_ERR_TIMEOUT", case
        assert time.perf_counter() - t0 < 30.0
        assert wt.mpq_check(P(ws), s) == 0      # reported once, then cleared
    # the default library still computes
    x, w = rand_i8(mpq, 3, 700, 1), rand_i8(mpq, 300, 700, 2)
    want = product64(x, w)
    assert_close(mpq.i8_linear(x, w), want, 3.01 * u * want.abs())
