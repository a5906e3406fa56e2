"""How many bits of a gradient enter the 8-bit integer layers' backward products.

A scaled gradient g (fp32) is rounded to 11 bits, off by at most half a step,
F16 = 2^-11 of its size, or by FLOOR = 2^-39 of its token's largest where it is
more than 28 powers of two below that one (fp16's last step, 2^-24, halved,
against a largest value of at least 2^14).  Codes are exact, the sum of n fp32
terms is off by at most 2 n u times the sum of their magnitudes, and the result
is rounded to bf16 once.
"""
import pytest

from test_gpu_i8 import B16, TINY, assert_close, gate64, gen, grads64, hat, mpq, product64, rand_i8, u  # noqa: F401

pytestmark = pytest.mark.gpu

F16 = 2.0 ** -11
FLOOR = 2.0 ** -39


def bounds(parts, n):
    """The sum of (scaled gradients, their tolerance, codes) products and its tolerance."""
    want, tol = 0, 0
    top = 0
    for g, _, _ in parts:
        top = g.abs().amax(1, keepdim=True).clamp_min(0 if isinstance(top, int) else top)
    for g, tg, q in parts:
        want = want + g @ q
        tol = tol + ((F16 + u) * g.abs() + tg + FLOOR * top + 2 * n * u * g.abs()) @ q.abs()
    return want, tol * 1.01 + B16 * want.abs() + TINY


TOKENS = [17, 33, 64, 65, 128, 129, 300]


@pytest.mark.parametrize("N", [1, 2, 5, 13, 200])
@pytest.mark.parametrize("M", TOKENS)
def test_linear_terms(mpq, M, N):
    import torch
    w = rand_i8(mpq, N, 300, 5, 1e-3)
    dy = (torch.randn(M, N, generator=gen(6), device="cuda") * 0.1).to(torch.bfloat16)
    g = dy.double() * w.scales.double()
    assert_close(mpq.i8_linear_backward(w, dy), *bounds([(g, u * g.abs(), w.codes.double())], N))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("F", [1, 3, 70])
@pytest.mark.parametrize("M", TOKENS)
def test_gated_terms(mpq, M, F, act):
    import torch
    K = 150
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x, wg, wu = rand_i8(mpq, M, K, 1), rand_i8(mpq, F, K, 2, sc), rand_i8(mpq, F, K, 3, sc)
    dh = (torch.randn(M, F, generator=gen(4), device="cuda") * 0.1).to(torch.bfloat16)
    wdg, wdu, tg, tu = grads64(act, x, wg, wu, dh)
    sg, su = wg.scales.double(), wu.scales.double()
    want, tol = bounds([(wdg * sg, tg * sg + u * (wdg * sg).abs(), wg.codes.double()),
                        (wdu * su, tu * su + u * (wdu * su).abs(), wu.codes.double())], 2 * F)
    assert_close(mpq.i8_gated_backward(x, wg, wu, dh, act=act)[0], want, tol)


@pytest.mark.parametrize("M", [17, 64, 140, 600])
def test_error_is_the_rounding_of_the_result(mpq, M):
    """Over many terms: the operand's roundings (at most F16 / sqrt(3) rms = 0.00028)
    add to the result's own (2^-8 / sqrt(3) / ~1.3 rms = 0.0017) in squares, 1.4 %
    at most; 5 % are allowed."""
    import torch
    N, K = 1000, 700
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x, wg, wu = rand_i8(mpq, M, K, 1), rand_i8(mpq, N, K, 2, sc), rand_i8(mpq, N, K, 3, sc)
    dy = torch.randn(M, N, generator=gen(4), device="cuda").to(torch.bfloat16)

    def check(dx, want):
        alone = torch.linalg.norm(want.to(torch.bfloat16).double() - want)
        assert float(torch.linalg.norm(dx.double() - want)) <= 1.05 * float(alone)
    check(mpq.i8_linear_backward(wg, dy), dy.double() @ hat(wg))
    wdg, wdu, _, _ = grads64("silu", x, wg, wu, dy)
    check(mpq.i8_gated_backward(x, wg, wu, dy)[0], wdg @ hat(wg) + wdu @ hat(wu))


@pytest.mark.parametrize("M", [1, 5, 16, 17, 40, 140])
def test_wide_ranges(mpq, M):
    """Tokens of very different sizes, zero ones, and values far below their
    token's largest where the codes of that one are zero."""
    import torch
    N, K = 130, 100
    w = rand_i8(mpq, N, K, 5)
    w.codes[7, :50] = 0
    w.codes[90, 25:] = 0
    e = torch.arange(M, device="cuda") * 37 % 121 - 60           # tokens from 2^-60 to 2^60
    dy = torch.randn(M, N, generator=gen(6), device="cuda")
    dy[:, 7] *= 2.0 ** 20
    dy[:, 90] *= 2.0 ** 24
    dy[M // 2] *= torch.randint(0, 2, (N,), generator=gen(7), device="cuda") * 2.0 ** -30 + 2.0 ** -10
    dy = torch.ldexp(dy, e[:, None]).to(torch.bfloat16)
    if M > 4:
        dy[3] = 0
    g = dy.double() * w.scales.double()
    want, tol = bounds([(g, u * g.abs(), w.codes.double())], N)
    dx = mpq.i8_linear_backward(w, dy)
    assert_close(dx, want, tol)
    # the ends of fp32: the largest finite gradients, and ones at and below the smallest normal number
    w.scales.fill_(1.0)
    for p in (110, -112, -126, -133, 126):
        dy = torch.ldexp((torch.rand(M, N, generator=gen(8), device="cuda") + 0.5), torch.tensor(p, device="cuda"))
        dy = dy.to(torch.bfloat16)
        if p == 126:
            w.codes.sign_()
        q = w.codes.double()
        want, tol = bounds([(dy.double(), 0 * dy.double(), q)], N)
        dx = mpq.i8_linear_backward(w, dy)
        # fp32 sums may pass the largest number on their way; a sum that does not, has its value
        sure = dy.double().abs() @ q.abs() < 3e38
        step = 2.0 ** -133 + N * 2.0 ** -149     # bf16's smallest step, and fp32's at every term
        assert_close(dx[sure], want[sure], tol[sure] - TINY + step)


@pytest.mark.parametrize("M,N", [(1, 8191), (1, 8193), (3, 70001), (16, 131071), (1, 400000), (40, 33000), (149, 33000),
                                 (200, 40003)])
def test_long_tokens(mpq, M, N):
    """Tokens of more columns than a block, or a cluster of blocks, keeps; the
    largest value at either end."""
    import torch
    w = rand_i8(mpq, N, 5, 5, 1e-3)
    for odd in (0, 1):
        dy = (torch.randn(M, N + odd, generator=gen(6), device="cuda") * 0.1).to(torch.bfloat16)[:, odd:]
        for at in (0, N - 1):
            dy[M - 1, at] = 300.0
        g = dy.double() * w.scales.double()
        dx = mpq.i8_linear_backward(w, dy)
        assert_close(dx, *bounds([(g, u * g.abs(), w.codes.double())], N))
