"""The bounded waits of the 8-bit integer kernels, made to run out without
faulting anything, as in test_gpu_timeout.py: the wait-test library's producers
arm their barriers without a copy and its waits give up after 2 ms.  Each call
must return, report MPQ_ERR_TIMEOUT through mpq_check and leave the context
usable."""
import ctypes
import time

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_wise_mixed_b200 import _lib, build
    build.build()
    wt = _lib.load(build.build_wait_test())
    import block_wise_mixed_b200 as m
    return m, _lib, wt


# few tokens (the streaming kernel), many (the two-SM tiles)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_waits_run_out(libs, M):
    import torch
    mpq, _lib, wt = libs
    F, K = 700, 1000
    g = torch.Generator(device="cuda").manual_seed(M)
    x, wg, wu = (mpq.i8_quantize(torch.randn(n, K, generator=g, device="cuda")) for n in (M, F, F))
    dh = torch.randn(M, F, generator=g, device="cuda").to(torch.bfloat16)
    h = torch.empty(M, F, device="cuda")
    dg, du = (torch.empty(M, F, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    dx = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    r, P = ctypes.byref, lambda t: ctypes.c_void_p(t.data_ptr())
    s = _lib._stream()
    ws = torch.zeros(wt.mpq_i8_gated_backward_workspace_size(M, F, K), dtype=torch.uint8, device="cuda")
    w = (P(ws), ws.numel(), s)
    calls = [
        lambda: wt.mpq_i8_linear(r(x.c), r(wg.c), P(h), 0, F, *w),
        lambda: wt.mpq_i8_gated(r(x.c), r(wg.c), r(wu.c), 0, P(h), 0, F, *w),
        lambda: wt.mpq_i8_linear_backward(r(wg.c), P(dh), M, F, P(dx), K, *w),
        lambda: wt.mpq_i8_gated_backward(r(x.c), r(wg.c), r(wu.c), 0, P(dh), F, P(dg), P(du), F, P(dx), K, *w),
    ]
    for call in calls:
        ws.zero_()
        t0 = time.perf_counter()
        assert call() == 0
        assert _lib.STATUS[wt.mpq_check(P(ws), s)] == "MPQ_ERR_TIMEOUT"
        assert time.perf_counter() - t0 < 30.0
        assert wt.mpq_check(P(ws), s) == 0      # reported once, then cleared
    # the default library still computes
    y = mpq.i8_linear(x, wg)
    want = (x.codes.double() @ wg.codes.double().t()) * wg.scales.double() * x.scales.double()[:, None]
    assert bool(((y.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all())
