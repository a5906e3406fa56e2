"""Every way that the 8-bit integer calls hand out their work (i8_shapes.py), and
the two-SM kernels over many columns, against the formulas in 64 bits with the
tolerances of test_gpu_i8.py and test_gpu_i8_gradients.py."""
import pytest

import i8_shapes
from test_gpu_i8 import (B16, TINY, assert_close, gate64, gen, grads64, guarded, guards_ok, mpq, product64,  # noqa: F401
                         rand_i8, same, u)
from test_gpu_i8_gradients import bounds

pytestmark = pytest.mark.gpu


def check_linear(mpq, M, N, K, odd):
    import torch
    x, w = rand_i8(mpq, M, K, 10 + M, 1e-2, extra=odd), rand_i8(mpq, N, K, 20 + N, 1e-3)
    want = product64(x, w)
    for dt, more in ((torch.float32, 0.0), (torch.bfloat16, B16)):
        buf, y = guarded(M, N, dt, odd)
        mpq.i8_linear(x, w, out=y)
        assert_close(y, want, (3 * u + more) * 1.001 * want.abs())
        assert guards_ok(buf, M, N)
        first = y.clone()
        assert same((mpq.i8_linear(x, w, out=y),), (first,))


def check_gated(mpq, M, F, K, odd):
    import torch
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x, wg, wu = rand_i8(mpq, M, K, 30 + M), rand_i8(mpq, F, K, 40 + F, sc, extra=odd), rand_i8(mpq, F, K, 50 + F, sc)
    a, b = product64(x, wg), product64(x, wu)
    for act in ("silu", "gelu_tanh"):
        t, g, _, _ = gate64(act, a)
        want = g * b
        for dt, more in ((torch.float32, 0.0), (torch.bfloat16, B16)):
            buf, h = guarded(M, F, dt, odd)
            mpq.i8_gated(x, wg, wu, act=act, out=h)
            assert_close(h, want, ((20 + 15 * t.abs()) * u + more) * 1.01 * want.abs() + TINY * (1 + b.abs()))
            assert guards_ok(buf, M, F)


def norm_ok(dx, want):
    import torch
    if want.numel() >= 64:
        assert float(torch.linalg.norm(dx.double() - want)) <= B16 * float(torch.linalg.norm(want))


def check_linear_backward(mpq, M, N, K, odd):
    import torch
    w = rand_i8(mpq, N, K, 60 + K % 97, 1e-3, extra=odd)
    dy = (torch.randn(M, N + odd, generator=gen(7), device="cuda") * 0.1).to(torch.bfloat16)[:, :N]
    buf, dx = guarded(M, K, torch.bfloat16, odd)
    mpq.i8_linear_backward(w, dy, out=dx)
    g = dy.double() * w.scales.double()
    want, tol = bounds([(g, u * g.abs(), w.codes.double())], N)
    assert_close(dx, want, tol)
    norm_ok(dx, want)
    assert guards_ok(buf, M, K)
    assert same((mpq.i8_linear_backward(w, dy),), (dx,))


def check_gated_backward(mpq, M, F, K, odd):
    import torch
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x, wg, wu = rand_i8(mpq, M, K, 70 + M), rand_i8(mpq, F, K, 80 + F, sc), rand_i8(mpq, F, K, 90 + F, sc, extra=odd)
    sg, su = wg.scales.double(), wu.scales.double()
    dh = (torch.randn(M, F + odd, generator=gen(8), device="cuda") * 0.1).to(torch.bfloat16)[:, :F]
    for act in ("silu", "gelu_tanh"):
        bufs = [guarded(M, n, torch.bfloat16, odd) for n in (K, F, F)]
        dx, dg, du = (b[1] for b in bufs)
        mpq.i8_gated_backward(x, wg, wu, dh, act=act, dx=dx, d_gate=dg, d_up=du)
        wdg, wdu, tg, tu = grads64(act, x, wg, wu, dh)
        assert_close(dg, wdg, tg * 1.01 + B16 * wdg.abs())
        assert_close(du, wdu, tu * 1.01 + B16 * wdu.abs())
        want, tol = bounds([(wdg * sg, tg * sg + u * (wdg * sg).abs(), wg.codes.double()),
                            (wdu * su, tu * su + u * (wdu * su).abs(), wu.codes.double())], 2 * F)
        assert_close(dx, want, tol)
        norm_ok(dx, want)
        for (buf, _), n in zip(bufs, (K, F, F)):
            assert guards_ok(buf, M, n)
        assert same(mpq.i8_gated_backward(x, wg, wu, dh, act=act), (dx, dg, du))


CHECK = {"linear": check_linear, "gated": check_gated, "linear_backward": check_linear_backward,
         "gated_backward": check_gated_backward}


@pytest.mark.parametrize("op,part,kernel,columns,how,M,N,K", i8_shapes.cases())
def test_plan(mpq, op, part, kernel, columns, how, M, N, K):
    assert i8_shapes.classes(mpq.i8_plan(op, M, N, K))[part] == (kernel, columns, how)
    CHECK[op](mpq, M, N, K, (M + N + K) % 4)


# the two-SM kernels' rings many times around, remainders in every direction
LONG = [("linear", 700, 5000, 3000), ("linear", 1025, 9000, 8190), ("gated", 600, 2000, 700), ("gated", 1300, 4001, 8190),
        ("gated", 120, 14000, 2000), ("gated_backward", 600, 2000, 700), ("gated_backward", 1300, 4001, 8190),
        ("gated_backward", 120, 14000, 2000), ("linear_backward", 1300, 8190, 4001)]
KERNELS = [("tile", 256), ("tile", 256), ("tile", 256), ("tile", 256), ("stream", 128), ("tile", 256), ("tile", 256),
           ("stream", 128), ("dx", 256)]


@pytest.mark.parametrize("case,kernel", list(zip(LONG, KERNELS)))
def test_long_columns(mpq, case, kernel):
    op, M, N, K = case
    plan = i8_shapes.classes(mpq.i8_plan(op, M, N, K))
    assert plan.get("product", plan.get("gradient"))[:2] == kernel
    CHECK[op](mpq, M, N, K, 3)
