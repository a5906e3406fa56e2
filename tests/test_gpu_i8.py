"""The 8-bit integer operators on the GPU against their formulas in 64 bits.

Tolerances count roundings: u = 2^-24 is half a step of fp32 relative to the
value, B16 = 2^-8 of bf16.  The int32 sums are exact, so

  product a     fl(fl(fl(acc) w.scale) x.scale): three roundings, 3 u |a|;
  act(a)        with a known to 3 u relative, t(a) to (3 * 3 + 6) u |t| (a cube
                and six roundings), sigmoid's relative error is at most the
                error of t plus 8 u (expf 2 ulp = 4 u, the reciprocal 2 ulp): in
                all below (20 + 15 |t|) u, which covers the product with b too;
  act'(a)       the same relative error on each of its two terms, and the
                curvature (at most 1.2 for both gates) times 3 u |a|;
  dx            every term's gradient is rounded to bf16 once (B16), the sum of
                n fp32 terms is off by at most 2 n u times the sum of their
                magnitudes, and the result is rounded once.
"""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
B16 = 2.0 ** -8
TINY = 1e-36   # below it fp32 is subnormal


@pytest.fixture(scope="module")
def mpq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_wise_mixed_b200 import build
    build.build()
    import block_wise_mixed_b200 as m
    return m


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def rand_i8(mpq, rows, cols, seed, scale=1.0, extra=0):
    """Random codes over the whole range, padding bytes and extra pitch filled
    with a value that would show in the sums, and positive scales."""
    import torch
    g = gen(seed)
    ld = (cols + 15) // 16 * 16 + 16 * extra
    buf = torch.full((rows, ld), 77, dtype=torch.int8, device="cuda")
    buf[:, :cols] = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    s = (torch.rand(rows, generator=g, device="cuda") + 0.5) * scale
    return mpq.i8_matrix(buf[:, :cols], s)


def hat(q):
    return q.codes.double() * q.scales.double()[:, None]


def product64(x, w):
    """x_hat w_hat^T with the sums over the integer codes, which 64 bits hold exactly."""
    return (x.codes.double() @ w.codes.double().t()) * w.scales.double() * x.scales.double()[:, None]


def guarded(rows, cols, dtype, extra):
    """An output view inside a larger buffer whose other elements must stay."""
    import torch
    buf = torch.full((rows + 2, cols + extra), 7.0, dtype=dtype, device="cuda")
    return buf, buf[1:rows + 1, :cols]


def guards_ok(buf, rows, cols):
    import torch
    m = torch.ones_like(buf, dtype=torch.bool)
    m[1:rows + 1, :cols] = False
    return bool((buf[m] == 7.0).all())


def assert_close(got, want, tol):
    import torch
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), "%d of %d off, worst %g of its tolerance" % (
        int(bad.sum()), bad.numel(), float((err / tol.clamp_min(1e-300)).max()))


def gate64(act, a):
    import torch
    c = (2.0 / np.pi) ** 0.5
    if act == "silu":
        t, dt = a, torch.ones_like(a)
    else:
        t, dt = 2 * c * (a + 0.044715 * a ** 3), 2 * c * (1 + 0.134145 * a * a)
    sig, cosig = torch.sigmoid(t), torch.sigmoid(-t)
    return t, a * sig, sig, a * sig * cosig * dt


# ------------------------------- rows ----------------------------------------
def quantize64(x):
    """Codes and scales by the definition (the scale in fp32, the quotient in 64 bits)."""
    import torch
    x = x.double()
    amax = x.abs().amax(1)
    s = (amax / 127).float().clamp_min(2.0 ** -126)
    s = torch.where(amax == 0, torch.ones_like(s), s)
    q = torch.round(x / s.double()[:, None])
    fin = torch.isfinite(amax)
    return torch.where(fin[:, None], q, torch.zeros_like(q)), torch.where(fin, s, torch.full_like(s, float("nan")))


ROWS = [(1, 1), (1, 7), (3, 16), (5, 33), (1, 4096), (2, 4095), (300, 130), (130, 1000), (150, 8192), (7, 14335),
        (160, 14336), (3, 16391), (2, 40000), (149, 33000), (2, 131071)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_quantize_codes_exact(mpq, rows, cols, dtype):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for extra in (0, 8, 3):    # aligned rows with and without a gap, rows at odd addresses
        big = torch.randn(rows, cols + extra, generator=gen(rows + cols), device="cuda").to(dt)
        x = big[:, :cols]
        q = mpq.i8_empty(rows, cols, "cuda")
        pad = torch.as_strided(q.codes, (rows, q.c.ld), (q.c.ld, 1))
        pad.fill_(55)
        assert mpq.i8_quantize(x, out=q) is q
        c64, s64 = quantize64(x)
        assert torch.equal(q.scales, s64)
        assert torch.equal(q.codes.double(), c64)
        assert bool((pad[:, cols:] == 55).all())
        # and back: one fp32 product, rounded once more to bf16
        v = q.codes.float() * q.scales[:, None]
        for odt in (torch.float32, torch.bfloat16):
            buf, out = guarded(rows, cols, odt, extra)
            mpq.i8_dequantize(q, out=out)
            assert torch.equal(out, v.to(odt)) and guards_ok(buf, rows, cols)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 7, 8, 9])
def test_quantize_narrow_rows(mpq, cols, dtype):
    """Rows that share their 16-byte blocks with other rows and with what lies
    before and behind the array (NaN here), from every offset."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for rows in (1, 2, 3, 9, 300):
        for off in range(9):
            buf = torch.full((rows * cols + 24,), float("nan"), dtype=dt, device="cuda")
            x = buf[off:off + rows * cols].view(rows, cols)
            x.copy_(torch.randn(rows, cols, generator=gen(rows + off), device="cuda"))
            q = mpq.i8_quantize(x)
            c64, s64 = quantize64(x)
            assert torch.equal(q.scales, s64) and torch.equal(q.codes.double(), c64)


def test_quantize_rounding_borders(mpq):
    """Quotients on, and a last place beside, every half step; scales over the
    whole range of fp32, subnormal values and zero rows among them."""
    import torch
    rows = []
    for e in (-149, -140, -133, -127, -126, -120, -60, -1, 0, 3, 100, 121):
        for top in (127.0, 100.0, 64.0, 127.0 * 1.2345678, 3.0000002):
            amax = np.float32(np.ldexp(top, e))
            if not np.isfinite(amax):
                continue
            s = max(np.float32(amax / np.float32(127)), np.float32(2.0 ** -126)) if amax else np.float32(1)
            h = np.arange(-127, 127, dtype=np.float64) + 0.5
            v = (h * np.float64(s)).astype(np.float32)
            v = np.concatenate([v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(-np.inf))])
            v = np.clip(v, -amax, amax).astype(np.float32)
            rows.append(np.concatenate([v, [amax, -amax, 0.0, -0.0]]).astype(np.float32))
    rows.append(np.zeros_like(rows[0]))
    x = torch.from_numpy(np.stack(rows)).cuda()
    for t in (x, x.to(torch.bfloat16)):
        q = mpq.i8_quantize(t)
        c64, s64 = quantize64(t)
        assert torch.equal(q.scales, s64)
        assert torch.equal(q.codes.double(), c64)


@pytest.mark.parametrize("cols", [5, 64, 1000, 20000])
def test_quantize_nonfinite_rows(mpq, cols):
    """A NaN or an infinity spoils its own row only: scale NaN, codes 0."""
    import torch
    x = torch.randn(6, cols, generator=gen(1), device="cuda")
    x[1, cols - 1] = float("nan")
    x[3, 0] = float("inf")
    x[4, cols // 2] = float("-inf")
    q = mpq.i8_quantize(x)
    c64, s64 = quantize64(x)
    assert torch.equal(torch.isnan(q.scales).cpu(), torch.tensor([0, 1, 0, 1, 1, 0], dtype=torch.bool))
    assert torch.equal(torch.nan_to_num(q.scales), torch.nan_to_num(s64))
    assert torch.equal(q.codes.double(), c64)
    w = rand_i8(mpq, 40, cols, 2)
    y = mpq.i8_linear(q, w)
    assert bool(torch.isnan(y[[1, 3, 4]]).all()) and bool(torch.isfinite(y[[0, 2, 5]]).all())


# ------------------------------ products --------------------------------------
MNK = [(1, 1, 1), (1, 5, 15), (2, 64, 16), (3, 130, 17), (1, 4096, 4096), (7, 300, 1000), (8, 1024, 8192),
       (15, 129, 127), (16, 128, 128), (17, 127, 129), (31, 1000, 333), (32, 2048, 512), (33, 257, 640),
       (63, 96, 2000), (64, 4096, 256), (65, 511, 384), (100, 1371, 1001), (127, 640, 1024), (128, 1027, 4095),
       (129, 512, 512), (130, 4096, 1024), (200, 1371, 2003), (255, 255, 255), (256, 256, 256), (257, 257, 257),
       (300, 5000, 768), (511, 2000, 1500), (512, 4096, 4096), (1000, 1000, 100), (2048, 1024, 1111),
       (4, 70, 131071), (300, 100, 131071)]


@pytest.mark.parametrize("M,N,K", MNK)
def test_linear(mpq, M, N, K):
    import torch
    x, w = rand_i8(mpq, M, K, 10 + M, 1e-2, extra=M % 3), rand_i8(mpq, N, K, 20 + N, 1e-3, extra=N % 2)
    want = product64(x, w)
    for dt, tol in ((torch.float32, 3 * u), (torch.bfloat16, 3 * u + B16)):
        for extra in (0, 8, 5):
            buf, y = guarded(M, N, dt, extra)
            mpq.i8_linear(x, w, out=y)
            assert_close(y, want, tol * 1.001 * want.abs())
            assert guards_ok(buf, M, N)


# (operator, tokens, channels, columns): tile counts for each way that work is
# handed out -- clusters of 2 to 8 pieces, whole rounds and cut remainders, equal
# runs over the last round -- in the products and in the gradients
WORK = [("linear", 1, 9000, 2048), ("linear", 3, 5000, 4096), ("linear", 2, 4000, 8192), ("linear", 5, 3000, 8192),
        ("linear", 20, 2500, 4096), ("linear", 1, 1700, 4096), ("linear", 40, 900, 8192), ("linear", 100, 1000, 4096),
        ("linear", 1, 21504, 4096), ("linear", 2, 9728, 16384), ("linear", 16, 19100, 6000), ("gated", 1, 9728, 8192),
        ("gated", 30, 1000, 4096), ("gated", 9, 20900, 4096), ("gated", 90, 2000, 2048),
        ("linear_backward", 16, 8192, 28672), ("linear_backward", 16, 8192, 512), ("linear_backward", 40, 5000, 900),
        ("linear_backward", 600, 12000, 6656), ("linear_backward", 100, 3000, 20000), ("gated_backward", 20, 3000, 700)]


@pytest.mark.parametrize("op,M,N,K", WORK)
def test_work_distribution(mpq, op, M, N, K):
    import torch
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x, wg = rand_i8(mpq, M, K, 1), rand_i8(mpq, N, K, 2, sc)
    wu = rand_i8(mpq, N, K, 3, sc) if "gated" in op else None
    dh = (torch.randn(M, N, generator=gen(4), device="cuda") * 0.1).to(torch.bfloat16)
    call = {"linear": lambda: (mpq.i8_linear(x, wg),), "gated": lambda: (mpq.i8_gated(x, wg, wu, ydtype=mpq.Y_F32),),
            "linear_backward": lambda: (mpq.i8_linear_backward(wg, dh),),
            "gated_backward": lambda: mpq.i8_gated_backward(x, wg, wu, dh)}[op]
    got = call()
    if op == "linear":
        want = product64(x, wg)
        assert_close(got[0], want, 3.01 * u * want.abs())
    elif op == "gated":
        a, b = product64(x, wg), product64(x, wu)
        t, g, _, _ = gate64("silu", a)
        assert_close(got[0], g * b, (20 + 15 * t.abs()) * u * 1.01 * (g * b).abs() + TINY * (1 + b.abs()))
    elif op == "linear_backward":
        assert_dx(got[0], *dx64([(dh.double(), u * dh.double().abs(), hat(wg))], N))
    else:
        wdg, wdu, tg, tu = grads64("silu", x, wg, wu, dh)
        assert_dx(got[0], *dx64([(wdg, tg, hat(wg)), (wdu, tu, hat(wu))], 2 * N))
    for _ in range(3):
        assert same(call(), got)


def test_linear_extreme_sums(mpq):
    """Sums next to the ends of int32 (every code -128 at the longest row), and
    scales whose product with the sum leaves fp32 only if the result does."""
    import torch
    K = 131071
    x, w = rand_i8(mpq, 5, K, 1), rand_i8(mpq, 9, K, 2)
    x.codes.fill_(-128)
    w.codes.fill_(-128)
    w.codes[3:] = 127
    x.scales.copy_(torch.tensor([1.0, 1e-30, 1e25, 2.0 ** -100, 0.0]))
    w.scales.copy_(torch.tensor([1e-3] * 4 + [1e-9] * 5))
    y = mpq.i8_linear(x, w)
    want = product64(x, w)
    assert_close(y, want, 4 * u * want.abs())


GATED = [(1, 1, 1), (1, 96, 64), (1, 1371, 1001), (5, 128, 200), (16, 256, 512), (17, 130, 129), (40, 1000, 1000),
         (64, 700, 256), (100, 257, 384), (128, 512, 640), (129, 1371, 500), (200, 1371, 2003), (256, 128, 1024),
         (257, 129, 300), (512, 1024, 512), (700, 333, 777)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated(mpq, M, F, K, act):
    import torch
    # pre-activations of a few units, as a model's are
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x = rand_i8(mpq, M, K, 30 + M, 1.0, extra=1)
    wg, wu = rand_i8(mpq, F, K, 40 + F, sc, extra=F % 2), rand_i8(mpq, F, K, 50 + F, sc)
    a, b = product64(x, wg), product64(x, wu)
    t, g, _, _ = gate64(act, a)
    want = g * b
    rel = (20 + 15 * t.abs()) * u
    for dt, more in ((torch.float32, 0.0), (torch.bfloat16, B16)):
        for extra in (0, 3):
            buf, h = guarded(M, F, dt, extra)
            mpq.i8_gated(x, wg, wu, act=act, out=h)
            assert_close(h, want, (rel + more) * 1.01 * want.abs() + TINY * (1 + b.abs()))
            assert guards_ok(buf, M, F)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_extreme(mpq, act):
    """Pre-activations far out on both sides, zero, and beyond fp32."""
    import torch
    M, F, K = 12, 40, 32
    x, wg, wu = rand_i8(mpq, M, K, 1), rand_i8(mpq, F, K, 2), rand_i8(mpq, F, K, 3)
    x.codes.fill_(1)
    wg.codes[: F // 2] = 1
    wg.codes[F // 2:] = -1
    x.scales.copy_(torch.tensor([0.0, 1e-20, 1e-3, 0.1, 1, 3, 10, 30, 1e3, 1e10, 1e15, float("nan")]))
    wg.scales.fill_(1.0)
    h = mpq.i8_gated(x, wg, wu, act=act, ydtype=mpq.Y_F32)
    a, b = product64(x, wg), product64(x, wu)
    t, g, _, _ = gate64(act, a)
    want = (g * b)[:-1]
    # t's error is relative, but where |t| > 110 the gate is 0 or 1 in fp32 whatever the error
    rel = (20 + 15 * t[:-1].abs().clamp_max(110)) * u
    assert_close(h[:-1], want, rel * want.abs() + 1e-30 * (1 + b[:-1].abs()))
    assert bool(torch.isnan(h[-1]).all())


# ------------------------------ gradients -------------------------------------
def grads64(act, x, wg, wu, dh):
    a, b = product64(x, wg), product64(x, wu)
    t, g, sig, curve = gate64(act, a)
    dh = dh.double()
    d_up = dh * g
    d_gate = dh * b * (sig + curve)
    rel = (20 + 15 * t.abs()) * u
    tol_up = rel * d_up.abs() + TINY
    tol_gate = (dh * b).abs() * (rel * (sig + curve.abs()) + 1.2 * 3 * u * a.abs()) + 5 * u * d_gate.abs() + TINY
    return d_gate, d_up, tol_gate, tol_up


def dx64(parts, n):
    """Sum of (gradient, its tolerance, dequantized weights) products, with the
    tolerance of the bf16 products."""
    want, tol = 0, 0
    for d, td, w in parts:
        want = want + d @ w
        tol = tol + td @ w.abs() + (B16 + 2 * n * u) * (d.abs() @ w.abs())
    return want, tol * 1.01 + B16 * want.abs() + TINY


def assert_dx(dx, want, tol):
    import torch
    assert_close(dx, want, tol)
    # two roundings to bf16 of at most 2^-8 / sqrt(3) rms each
    if want.numel() >= 64:
        assert float(torch.linalg.norm(dx.double() - want)) <= B16 * float(torch.linalg.norm(want))


LB = [(1, 1, 1), (1, 130, 64), (1, 4096, 4096), (2, 17, 200), (5, 1000, 257), (16, 8192, 512), (17, 64, 1000),
      (33, 333, 128), (64, 1371, 1001), (65, 200, 129), (100, 4096, 256), (128, 512, 2000), (129, 700, 384),
      (256, 256, 256), (257, 1001, 513), (300, 64, 5000), (512, 4096, 1024), (1000, 130, 300), (6, 33, 131071)]


@pytest.mark.parametrize("M,N,K", LB)
def test_linear_backward(mpq, M, N, K):
    import torch
    w = rand_i8(mpq, N, K, 60 + K % 97, 1e-3, extra=N % 2)
    for extra in (0, 3):
        dy = (torch.randn(M, N + extra, generator=gen(7), device="cuda") * 0.1).to(torch.bfloat16)[:, :N]
        buf, dx = guarded(M, K, torch.bfloat16, extra)
        mpq.i8_linear_backward(w, dy, out=dx)
        want, tol = dx64([(dy.double(), u * dy.double().abs(), hat(w))], N)
        assert_dx(dx, want, tol)
        assert guards_ok(buf, M, K)


@pytest.mark.parametrize("M", [16, 64, 128, 512])
def test_linear_backward_cold_weights(mpq, M):
    """Long runs of code copies that come from HBM at their own pace (five
    weight matrices in turn, none left in the cache), every result the same
    bits as the first round's and that one within its tolerance."""
    import torch
    N, K = 2048, 14336
    ws = [rand_i8(mpq, N, K, s, 1e-3) for s in range(5)]
    dy = (torch.randn(M, N, generator=gen(7), device="cuda") * 0.1).to(torch.bfloat16)
    first = [mpq.i8_linear_backward(w, dy) for w in ws]
    for dx, w in zip(first, ws):
        want, tol = dx64([(dy.double(), u * dy.double().abs(), hat(w))], N)
        assert_dx(dx, want, tol)
    space = torch.zeros(mpq.i8_linear_backward_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        again = [mpq.i8_linear_backward(w, dy, ws=space) for w in ws]
        assert same(again, first)
    mpq.check(space)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", [(1, 1, 1), (1, 96, 64), (3, 1371, 200), (16, 256, 512), (61, 1371, 1001),
                                   (64, 130, 129), (128, 512, 300), (129, 700, 640), (256, 300, 256), (300, 257, 1000),
                                   (520, 1024, 512)])
def test_gated_backward(mpq, M, F, K, act):
    import torch
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x = rand_i8(mpq, M, K, 70 + M, 1.0, extra=1)
    wg, wu = rand_i8(mpq, F, K, 80 + F, sc), rand_i8(mpq, F, K, 90 + F, sc, extra=1)
    for extra in (0, 3):
        dh = (torch.randn(M, F + extra, generator=gen(8), device="cuda") * 0.1).to(torch.bfloat16)[:, :F]
        bufs = [guarded(M, n, torch.bfloat16, extra) for n in (K, F, F)]
        dx, dg, du = (b[1] for b in bufs)
        mpq.i8_gated_backward(x, wg, wu, dh, act=act, dx=dx, d_gate=dg, d_up=du)
        wdg, wdu, tg, tu = grads64(act, x, wg, wu, dh)
        assert_close(dg, wdg, tg * 1.01 + B16 * wdg.abs())
        assert_close(du, wdu, tu * 1.01 + B16 * wdu.abs())
        want, tol = dx64([(wdg, tg, hat(wg)), (wdu, tu, hat(wu))], 2 * F)
        assert_dx(dx, want, tol)
        for (buf, _), n in zip(bufs, (K, F, F)):
            assert guards_ok(buf, M, n)
    # without the pre-activation gradients: the same dx, bit for bit
    from block_wise_mixed_b200 import _lib
    dx2 = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(mpq.i8_gated_backward_workspace_size(M, F, K), dtype=torch.uint8, device="cuda")
    st = _lib.lib().mpq_i8_gated_backward(ctypes.byref(x.c), ctypes.byref(wg.c), ctypes.byref(wu.c),
                                          _lib._ACTS[act], dh.data_ptr(), dh.stride(0) if M > 1 else F + 3, None, None,
                                          0, dx2.data_ptr(), K, ws.data_ptr(), ws.numel(), _lib._stream())
    assert st == 0 and torch.equal(dx2, dx)


@pytest.mark.parametrize("M,N,K", [(1, 1350, 25), (2, 1024, 64), (4, 5000, 3), (16, 4096, 300), (1, 8192, 4096), (7, 100, 7)])
def test_few_tokens_carry_two_parts(mpq, M, N, K):
    """Up to 16 tokens the scaled gradient is a sum of two bf16 parts, so it is
    off by at most half a step of the second, 2^-16 of its size; what is left is
    the result's own rounding and the fp32 sums."""
    import torch
    w = rand_i8(mpq, N, K, 5, 1e-3)
    dy = (torch.randn(M, N, generator=gen(6), device="cuda") * 0.1).to(torch.bfloat16)
    want = dy.double() @ hat(w)
    mag = dy.double().abs() @ hat(w).abs()
    assert_close(mpq.i8_linear_backward(w, dy), want, (B16 * B16 + u + 2 * N * u) * mag + B16 * want.abs())


def test_gradients_against_differences(mpq):
    """dx along random directions against central differences of the block in
    64 bits (x_hat is what the codes stand for)."""
    import torch
    M, F, K = 5, 70, 90
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x, wg, wu = rand_i8(mpq, M, K, 1), rand_i8(mpq, F, K, 2, sc), rand_i8(mpq, F, K, 3, sc)
    dh = (torch.randn(M, F, generator=gen(4), device="cuda") * 0.1).to(torch.bfloat16)
    for act in ("silu", "gelu_tanh"):
        dx, dg, du = mpq.i8_gated_backward(x, wg, wu, dh, act=act)

        def loss(xh):
            a, b = xh @ hat(wg).t(), xh @ hat(wu).t()
            return (dh.double() * gate64(act, a)[1] * b).sum()
        _, tol = dx64([(dg.double(), 0 * dg.double(), hat(wg)), (du.double(), 0 * du.double(), hat(wu))], 2 * F)
        for i in range(4):
            v = torch.randn(M, K, generator=gen(20 + i), device="cuda").double()
            h = 1e-4
            diff = (loss(hat(x) + h * v) - loss(hat(x) - h * v)) / (2 * h)
            assert abs(float((dx.double() * v).sum() - diff)) <= float((tol * 2 * v.abs()).sum())
    w = rand_i8(mpq, F, K, 5, 1e-2)
    dy = (torch.randn(M, F, generator=gen(6), device="cuda")).to(torch.bfloat16)
    dx = mpq.i8_linear_backward(w, dy)
    _, tol = dx64([(dy.double(), 0 * dy.double(), hat(w))], F)
    v = torch.randn(M, K, generator=gen(9), device="cuda").double()
    diff = (dy.double() * (v @ hat(w).t())).sum()      # the layer is linear in x
    assert abs(float((dx.double() * v).sum() - diff)) <= float((tol * v.abs()).sum())


def test_nonfinite_gradients_stay_in_their_rows(mpq):
    import torch
    M, F, K = 140, 200, 150
    x, wg, wu = rand_i8(mpq, M, K, 1, 0.01), rand_i8(mpq, F, K, 2, 0.01), rand_i8(mpq, F, K, 3, 0.01)
    dh = torch.ones(M, F, device="cuda", dtype=torch.bfloat16)
    dh[3, 199] = float("nan")
    dh[135, 0] = float("inf")
    dx, dg, du = mpq.i8_gated_backward(x, wg, wu, dh)
    bad = ~torch.isfinite(dx).all(1)
    assert bad.nonzero().flatten().tolist() == [3, 135]
    dxl = mpq.i8_linear_backward(wg, dh)
    assert (~torch.isfinite(dxl).all(1)).nonzero().flatten().tolist() == [3, 135]


@pytest.mark.parametrize("M", [1, 5, 16, 17, 140])
def test_infinite_gradients_keep_their_sign(mpq, M):
    """inf times a code is an infinity of the code's sign (NaN for a code of 0),
    for few tokens, whose gradients go in two parts, as for many."""
    import torch
    N, K = 200, 150
    w = rand_i8(mpq, N, K, 2, 0.01)
    w.codes[7, 5] = 0
    dy = torch.ones(M, N, device="cuda", dtype=torch.bfloat16)
    dy[0, 7] = float("inf")
    dy[M - 1, 100] = float("-inf")
    want = (dy.double() * w.scales.double()) @ w.codes.double()
    dx = mpq.i8_linear_backward(w, dy)
    bad = ~torch.isfinite(want)
    assert int(bad.sum()) >= K and torch.equal(~torch.isfinite(dx), bad)
    assert torch.equal(dx.double().nan_to_num(0.0, 1.0, -1.0)[bad], want.nan_to_num(0.0, 1.0, -1.0)[bad])
    # and through the gated block
    x, wg = rand_i8(mpq, M, K, 3, 0.01), rand_i8(mpq, N, K, 4, 0.01)
    dx, d_gate, d_up = mpq.i8_gated_backward(x, wg, w, dy)
    want = (d_gate.double() * wg.scales.double()) @ wg.codes.double() + (d_up.double() * w.scales.double()) @ w.codes.double()
    bad = ~torch.isfinite(want)
    assert int(bad.sum()) >= K and torch.equal(~torch.isfinite(dx), bad)
    assert torch.equal(dx.double().nan_to_num(0.0, 1.0, -1.0)[bad], want.nan_to_num(0.0, 1.0, -1.0)[bad])


# ------------------------- a block, end to end --------------------------------
def test_feed_forward_block(mpq):
    """quantize -> gated -> quantize -> linear, each step checked against its
    formula on the codes that the step before produced; and the gated output
    straight into a mixed-precision linear layer, as the library's layers are
    used together."""
    import torch
    from block_wise_mixed_b200 import synth
    D, F = 512, 1408
    for M in (1, 9, 150):
        h0 = torch.randn(M, D, generator=gen(M), device="cuda").to(torch.bfloat16)
        wg, wu, wd = (mpq.i8_quantize(torch.randn(n, k, generator=gen(s), device="cuda") * 0.05)
                      for n, k, s in ((F, D, 1), (F, D, 2), (D, F, 3)))
        x = mpq.i8_quantize(h0)
        h = mpq.i8_gated(x, wg, wu)
        a, b = product64(x, wg), product64(x, wu)
        t, g, _, _ = gate64("silu", a)
        assert_close(h, g * b, ((20 + 15 * t.abs()) * u + B16) * (g * b).abs() + TINY)
        hq = mpq.i8_quantize(h)
        c64, s64 = quantize64(h)
        assert torch.equal(hq.codes.double(), c64) and torch.equal(hq.scales, s64)
        y = mpq.i8_linear(hq, wd)
        want = product64(hq, wd)
        assert_close(y, want, 3.01 * u * want.abs())
        # the block and back through its own gradients
        dy = torch.randn(M, D, generator=gen(5), device="cuda").to(torch.bfloat16)
        dh = mpq.i8_linear_backward(wd, dy)
        dx, dg, du = mpq.i8_gated_backward(x, wg, wu, dh)
        wdg, wdu, tg, tu = grads64("silu", x, wg, wu, dh)
        want, tol = dx64([(wdg, tg, hat(wg)), (wdu, tu, hat(wu))], 2 * F)
        assert_dx(dx, want, tol)
        # mixed-precision layers around it: fp32 product -> quantize, bf16 h -> linear
        L = synth.make_layer("down", D, F, 3.0, 5, "random")
        P = mpq.pack(torch.from_numpy(L.W.view(np.int16)).cuda(), L.bits, L.row_perm, L.col_perm)
        y2 = mpq.linear(P, h)
        yq = mpq.i8_quantize(y2)
        c64, s64 = quantize64(y2)
        assert torch.equal(yq.codes.double(), c64) and torch.equal(yq.scales, s64)


# --------------------- streams, graphs, workspaces ----------------------------
def ops(mpq, M, F, K, seed):
    """(name, call(ws)) of every product on fixed inputs; a call returns its outputs."""
    import torch
    sc = 3.0 / (74.0 * 74.0 * K ** 0.5)
    x = rand_i8(mpq, M, K, seed)
    wg, wu = rand_i8(mpq, F, K, seed + 1, sc), rand_i8(mpq, F, K, seed + 2, sc)
    dh = torch.randn(M, F, generator=gen(seed + 3), device="cuda").to(torch.bfloat16)
    return [("linear", lambda **k: (mpq.i8_linear(x, wg, **k),)), ("gated", lambda **k: (mpq.i8_gated(x, wg, wu, **k),)),
            ("gated_backward", lambda **k: mpq.i8_gated_backward(x, wg, wu, dh, **k)),
            ("linear_backward", lambda **k: (mpq.i8_linear_backward(wg, dh, **k),))]


SHAPES = [(1, 1371, 1001), (9, 2000, 4096), (70, 300, 900), (200, 1371, 2003), (600, 1024, 512)]


def same(a, b):
    import torch
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_one_workspace_for_all_calls(mpq):
    """One zeroed workspace through all operators and shapes in any order gives
    what fresh workspaces give, and the same bits again on a second round."""
    import torch
    calls = [c for i, s in enumerate(SHAPES) for c in ops(mpq, *s, 100 * i)]
    fresh = [c() for _, c in calls]
    size = max(f(*s) for s in SHAPES for f in (mpq.i8_linear_workspace_size, mpq.i8_gated_workspace_size,
                                               mpq.i8_gated_backward_workspace_size,
                                               mpq.i8_linear_backward_workspace_size))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for order in (range(len(calls)), reversed(range(len(calls)))):
        for i in order:
            assert same(calls[i][1](ws=ws), fresh[i]), calls[i][0]
    mpq.check(ws)


@pytest.mark.parametrize("M,F,K", SHAPES)
def test_streams_and_graphs(mpq, M, F, K):
    """Another stream gives the same bits; so do two graphs that share one
    workspace, replayed in turn after their inputs changed in place."""
    import torch
    s = torch.cuda.Stream()
    for name, call in ops(mpq, M, F, K, 7):
        want = call()
        torch.cuda.synchronize()
        got = call(stream=s)
        s.synchronize()
        assert same(got, want), name
        with torch.cuda.stream(s):
            got = call()
        s.synchronize()
        assert same(got, want), name
    x = torch.randn(M, K, generator=gen(1), device="cuda").to(torch.bfloat16)
    wg, wu = rand_i8(mpq, F, K, 2, 1e-4), rand_i8(mpq, F, K, 3, 1e-4)
    dh = torch.randn(M, F, generator=gen(4), device="cuda").to(torch.bfloat16)
    q = mpq.i8_empty(M, K, "cuda")
    ws = torch.zeros(max(mpq.i8_gated_workspace_size(M, F, K), mpq.i8_gated_backward_workspace_size(M, F, K)),
                     dtype=torch.uint8, device="cuda")
    h = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    dx, dg, du = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (K, F, F))

    def fwd():
        mpq.i8_quantize(x, out=q)
        mpq.i8_gated(q, wg, wu, out=h, ws=ws)

    def bwd():
        mpq.i8_gated_backward(q, wg, wu, dh, dx=dx, d_gate=dg, d_up=du, ws=ws)
    graphs = []
    for f in (fwd, bwd):
        with torch.cuda.stream(s):
            f()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for rep in range(3):
        x.copy_(torch.randn(M, K, generator=gen(30 + rep), device="cuda"))
        dh.copy_(torch.randn(M, F, generator=gen(40 + rep), device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        q2 = mpq.i8_quantize(x)
        assert torch.equal(q2.codes, q.codes) and torch.equal(h, mpq.i8_gated(q2, wg, wu))
        assert same((dx, dg, du), mpq.i8_gated_backward(q2, wg, wu, dh))
    mpq.check(ws)


def test_weights_written_right_before(mpq):
    """Launches overlap the kernel before them: weights and activations
    quantized by the calls right before, again and again, are read complete."""
    import torch
    W = [torch.randn(2048, 1024, generator=gen(i), device="cuda") for i in range(3)]
    x = [torch.randn(8, 1024, generator=gen(9 + i), device="cuda") for i in range(3)]
    ref = [mpq.i8_linear(mpq.i8_quantize(x[i]), mpq.i8_quantize(W[i])) for i in range(3)]
    torch.cuda.synchronize()
    q, w = mpq.i8_empty(8, 1024, "cuda"), mpq.i8_empty(2048, 1024, "cuda")
    ws = torch.zeros(mpq.i8_linear_workspace_size(8, 2048, 1024), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(8, 2048, device="cuda") for _ in range(30)]
    for r in range(30):
        mpq.i8_quantize(W[r % 3], out=w)
        mpq.i8_quantize(x[r % 3], out=q)
        mpq.i8_linear(q, w, out=outs[r], ws=ws)
    for r in range(30):
        assert torch.equal(outs[r], ref[r % 3])


def test_binding_refuses_tensors(mpq):
    """Layouts, types and sizes that the calls do not take are refused, not read."""
    import torch
    x, w, w2 = rand_i8(mpq, 4, 64, 1), rand_i8(mpq, 8, 64, 2), rand_i8(mpq, 9, 64, 3)
    dy = torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)
    f = torch.zeros(4, 64, device="cuda")
    bad = [
        lambda: mpq.i8_quantize(f.t()), lambda: mpq.i8_quantize(f[:1].expand(4, 64)), lambda: mpq.i8_quantize(f.half()),
        lambda: mpq.i8_quantize(f, out=w), lambda: mpq.i8_quantize(f.double()),
        lambda: mpq.i8_matrix(x.codes[:, 1:], x.scales), lambda: mpq.i8_matrix(x.codes, x.scales[:3]),
        lambda: mpq.i8_matrix(x.codes, x.scales.double()),
        lambda: mpq.i8_matrix(torch.zeros(4, 20, device="cuda", dtype=torch.int8), x.scales),
        lambda: mpq.i8_linear(x, rand_i8(mpq, 8, 65, 4)), lambda: mpq.i8_linear(x, w, out=torch.zeros(4, 9, device="cuda")),
        lambda: mpq.i8_linear(x, w, out=torch.zeros(8, 4, device="cuda").t()), lambda: mpq.i8_linear(x.codes, w),
        lambda: mpq.i8_linear(x, w, out=torch.zeros(4, 8, device="cuda", dtype=torch.float16)),
        lambda: mpq.i8_linear(x, w, ws=torch.zeros(256, device="cuda", dtype=torch.uint8)),
        lambda: mpq.i8_linear(x, w, ws=torch.zeros(1 << 20, device="cuda", dtype=torch.uint8)[16:]),
        lambda: mpq.i8_gated(x, w, w2), lambda: mpq.i8_gated(x, w, w, act="relu"),
        lambda: mpq.i8_linear_backward(w, dy.float()), lambda: mpq.i8_linear_backward(w2, dy),
        lambda: mpq.i8_linear_backward(w, dy[:1].expand(4, 8)), lambda: mpq.i8_linear_backward(w, dy.t()),
        lambda: mpq.i8_gated_backward(x, w, w, dy[:3]), lambda: mpq.i8_gated_backward(x, w, w2, dy),
        lambda: mpq.i8_gated_backward(x, w, w, dy, d_gate=torch.zeros(4, 16, device="cuda", dtype=torch.bfloat16)[:, :8]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(mpq.MpqError):
            call()
            print("call %d was taken" % i)
    # empty batches are no-ops
    e = mpq.i8_quantize(torch.zeros(0, 64, device="cuda"))
    assert mpq.i8_linear(e, w).shape == (0, 8) and mpq.i8_gated(e, w, w).shape == (0, 8)
    assert mpq.i8_linear_backward(w, dy[:0]).shape == (0, 64)
    assert [t.shape for t in mpq.i8_gated_backward(e, w, w, dy[:0])] == [(0, 64), (0, 8), (0, 8)]
    assert mpq.i8_dequantize(e).shape == (0, 64)
    # and the calls above left nothing behind
    want = product64(x, w)
    assert_close(mpq.i8_linear(x, w), want, 4 * u * want.abs())


def test_two_streams_at_once(mpq):
    """Calls that overlap on two streams, each with its own workspace."""
    import torch
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [ops(mpq, *s, 11 * i) for i, s in enumerate(((5, 3000, 4096), (300, 1371, 1001)))]
    want = [[c() for _, c in calls] for calls in sets]
    torch.cuda.synchronize()
    spaces = [torch.zeros(64 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append([c(ws=spaces[i]) for _, c in sets[i]])
    torch.cuda.synchronize()
    for i in range(2):
        for rep in got[i]:
            assert all(same(a, b) for a, b in zip(rep, want[i]))
        mpq.check(spaces[i])


def test_offsets_beyond_32_bits(mpq):
    """Codes beyond 2^31 bytes and outputs beyond 2^31 elements."""
    import torch
    N, K, M = 140000, 16384, 3
    codes = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    rows = torch.tensor([0, 1, 131071, 131072, N - 2, N - 1], device="cuda")
    codes[rows] = torch.randint(-127, 128, (len(rows), K), generator=gen(1), device="cuda", dtype=torch.int8)
    w = mpq.i8_matrix(codes, torch.full((N,), 0.5, device="cuda"))
    x = rand_i8(mpq, M, K, 2)
    y = mpq.i8_linear(x, w)
    sel = codes[rows].double() * 0.5
    want = product64(x, mpq.i8_matrix(codes[rows], w.scales[rows]))
    assert_close(y[:, rows], want, 4 * u * want.abs())
    mask = torch.ones(N, dtype=torch.bool, device="cuda")
    mask[rows] = False
    assert bool((y[:, mask] == 0).all())
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    dy[:, rows] = 1.0
    dx = mpq.i8_linear_backward(w, dy)
    want, tol = dx64([(dy[:, rows].double(), 0 * dy[:, rows].double(), sel)], N)
    assert_dx(dx, want, tol)
    del codes, w, y, dy
    M, N, K = 70000, 32768, 32
    x, w = rand_i8(mpq, M, K, 3), rand_i8(mpq, N, K, 4)
    y = mpq.i8_linear(x, w, ydtype=mpq.Y_BF16)
    for m in (0, 65535, 65536, M - 1):
        want = product64(mpq.i8_matrix(x.codes[m:m + 1], x.scales[m:m + 1]), w)
        assert_close(y[m:m + 1], want, (4 * u + B16) * want.abs())


def test_largest_row_counts(mpq):
    """2^31 - 1 channels and 2^31 - 1 tokens: counts of tiles and last columns."""
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    R, K, E = 2 ** 31 - 1, 16, 300
    codes = torch.zeros((R, K), dtype=torch.int8, device="cuda")
    for i, part in enumerate((codes[:E], codes[-E:])):
        part.copy_(torch.randint(-127, 128, (E, K), generator=gen(i), device="cuda", dtype=torch.int8))
    big = mpq.i8_matrix(codes, torch.full((R,), 0.5, device="cuda"))
    ends = mpq.i8_matrix(torch.cat([codes[:E], codes[-E:]]), torch.full((2 * E,), 0.5, device="cuda"))
    one = rand_i8(mpq, 1, K, 2)
    want = product64(one, ends)

    def check(y, want, tol):   # a row of R values: zero but for its ends
        assert_close(torch.cat([y[:E], y[-E:]])[None].double(), want, tol)
        for i in range(E, R - E, 1 << 28):
            assert not bool(y[i:min(i + (1 << 28), R - E)].any())

    check(mpq.i8_linear(one, big, ydtype=mpq.Y_BF16)[0], want, (4 * u + B16) * want.abs())
    check(mpq.i8_linear(big, one, ydtype=mpq.Y_BF16)[:, 0], want, (4 * u + B16) * want.abs())
    h = mpq.i8_gated(one, big, big)[0]
    sig = torch.sigmoid(want)
    rel = (20 + 15 * want.abs().clamp_max(110)) * u + B16
    check(h, want * want * sig, rel * want * want * sig + 1e-30 * (1 + want.abs()))
    del h
    dy = torch.zeros((1, R), dtype=torch.bfloat16, device="cuda")
    for i, part in enumerate((dy[:, :E], dy[:, -E:])):
        part.copy_(torch.randn(1, E, generator=gen(5 + i), device="cuda"))
    dx = mpq.i8_linear_backward(big, dy)
    d = torch.cat([dy[:, :E], dy[:, -E:]], 1).double()
    want = d @ hat(ends)
    # (terms that are zero add without a rounding)
    assert_close(dx, want, (B16 * B16 + u + 4 * E * u) * (d.abs() @ hat(ends).abs()) + B16 * want.abs())
